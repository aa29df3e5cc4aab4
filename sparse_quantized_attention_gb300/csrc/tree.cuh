// tree.cuh -- speculative decoding over the 16-bit cache: argument bundles and what its kernels share.
#pragma once

#include "common.cuh"

namespace ffd {
namespace tree {

constexpr int kMaxNodes = FFD_TREE_MAX_NODES;
constexpr int kMaxPlace = 1 << 24;  // rotary positions are below
// Pages' time that an item counts for besides its pages when the pages of a batch are cut into equal ranges:
// what a CTA spends between two items. us without and with it: eight sequences of 500 to 8000 tokens, 8 heads, 25
// nodes 50.4 45.3; 32 sequences of 1000 to 9000, 2 heads, 8 nodes 43.4 40; four of 131072, 4 heads, 112 rows 176.8 173.3.
constexpr int kItemPages = 9;

// Pages of a CTA, at least, where CTAs share an item of np pages: a page takes 0.45 us and each CTA more about 0.06
// of the join, whose sum is least at a third of the square root. us by pages a CTA, 12 nodes of 8 heads: of 16
// pages 1 12.6, 2 12.5, 4 14.0; of 64 1 14.0, 3 12.8, 8 15.3; of 256 2 17.4, 5 15.3, 16 20.1; of 1024 8 22.7, 10
// 22.2, 24 26.8. Five pages take 11.7 one by one and 9.6 by a CTA alone, sixteen 12.5 and 15.5. Two tiles' records are
// twice as large, and their pages take twice the time too: 32 nodes of 8 heads, one KV head over 1024, 4096, 16384 and
// 65536 tokens, with half of these pages, these, and twice: 15.1 15.8 17.1, 17.6 17.4 20.0, 24.3 23.6 25.5, 38.1 34.7 41.1.
constexpr int kWholePages = 9;  // as many that one CTA takes all
__host__ __device__ inline int share_pages(int np) {
    if (np <= kWholePages) return np > 0 ? np : 1;
    return (int)ceilf(sqrtf((float)np) * (1.0f / 3.0f));
}

// Arguments of an append.
struct RopeArgs {
    int B, Hq, Hkv, P, max_blocks, T, each, rot, interleaved;
    int parts, per;  // warps of a token, rows of each
    float scale;
    int64_t q_stride, q_out_stride, k_stride, v_stride;  // elements
    const uint16_t *q, *k_new, *v_new;
    const float *inv_freq;
    const int32_t *places, *cu, *positions, *block_table;
    uint16_t *q_out, *k, *v;
    uint8_t *thumb, *resid;
    int *err;
};

// Arguments of a commit.
struct CommitArgs {
    int B, Hkv, P, max_blocks, T, each;
    const int64_t *draft, *target;
    const int32_t *parents, *cu, *seq_lens, *block_table;
    uint8_t *k, *v, *thumb, *resid;
    int32_t *path, *accepted, *new_lens;
    int64_t *next_token;
    int *err;
};

// Arguments of an attention call.
struct AttnArgs {
    int B, Hq, Hkv, G, P, max_blocks, max_q, total_q, window;
    int shares, groups, by_mask;  // as in Plan
    // ceil(2^32 / d) of small divisors d, 0 for 1
    uint32_t over_shares, over_groups, over_heads;
    int tile_nodes, item_nodes;  // of a tile of 128 rows, of an item
    int wide_out;     // out is aligned to 32 bytes
    uint32_t over_g;  // ceil(2^32 / G), too large by less than G / 2^32 of it (G > 1)
    int64_t q_stride;
    float factor;     // of scores, to log2 units
    const uint16_t *q, *k, *v;
    const uint8_t *keep_in;
    const int32_t *seq_lens, *cu_q, *block_table, *parents;
    uint16_t *out;
    float *lse;
    int *err;  // the workspace: error word first
    uint64_t wait_ns;
};

// Launch shape and workspace of an attention call (byte offsets behind the error word).
struct Plan {
    int tiles;  // of 128 rows that walk the cache together: 1 or 2
    int ctas;
    int shares; // equal shares that items may be dealt out in, 0: they may not
    int groups; // of a sequence's rows, at most
    int by_mask;  // whether a mask's kept blocks are counted, and shared out evenly
    size_t tickets, records, total;
};

// Sequence of row t and the row's place in it, by a whole warp: the offsets cu [B+1] are searched 32
// at a time (or rows are `each` a sequence when cu is null). False when the row belongs to nobody.
__device__ __forceinline__ bool row_of_warp(const int32_t *cu, int B, int each, int t, int lane, int &b,
                                            int &i) {
    if (!cu) {
        b = t / each;
        i = t - b * each;
        return true;
    }
    int lo = 0, hi = B;  // the largest b in [lo, hi) with cu[b] <= t
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + lane * step;
        const uint32_t below = __ballot_sync(0xffffffffu, lane == 0 || (at < hi && __ldg(cu + at) <= t));
        lo += (31 - __clz((int)below)) * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    b = lo;
    const int c = __ldg(cu + lo);
    i = t - c;
    return c >= 0 && c <= t && t < __ldg(cu + lo + 1);
}

}  // namespace tree
}  // namespace ffd
