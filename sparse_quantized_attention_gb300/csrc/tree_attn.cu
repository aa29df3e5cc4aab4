// tree_attn.cu -- attention of a tree of drafted tokens over the 16-bit cache on the fifth-generation
// tensor cores (ffd_tree_attention in ffd.h).
//
// The query rows of a (sequence, KV head), nq nodes x G heads, are taken a tile of 128 / G whole nodes, or two
// such tiles, at a time: an item is one such group of rows over the pages that any of them sees. The pages
// of all items, concatenated with what each item costs besides, are cut into equal contiguous ranges, one
// per CTA (one per SM). CTAs that share an item write their parts as records and join some of its channels each;
// the one in whose range it begins only where that is all it has: it may have another item to join. Page by
// page a CTA computes for each tile of 128 rows
//   S = Q K^T   (M 128, N 64, K 128; both operands in shared memory, S in tensor memory),
//   P = 2^(S - m) against a reference m that follows the row's maximum lazily: it is raised, and O rescaled,
//       only when a score passes it by 2^8,
//   O += P V    (M 128, N 128, K 64 a page; P in tensor memory over S, V in shared memory, O in tensor memory).
// P goes into its product as two numbers of the inputs' type, itself rounded and what that leaves out: one number
// would add an error as large as the output's own rounding (relative L2 1.7e-3 -> 2.4e-3 in bf16, 2.1e-4 -> 2.9e-4 in fp16).
// One tile has room for the second product: four of 131072 tokens, 112 rows 175 us with one part and with two, 32
// windows of 4096 99 and 99. Two tiles pay for it: four of 32768, 8 heads, 240 rows 110 and 131 us, eight ragged trees
// of 30 to 61 nodes 89 and 103, 96 blocks of 4 x 131072 with 25 nodes 31.2 and 33.8. Where there are more rows than two tiles take,
// the matrix unit is what bounds the call (2048 tokens over 32768: 729 and 947) and P has one part. Its rounding
// then counts on both sides: O is divided by the sum of the rounded numbers, so that the weights of V have the sum 1
// whatever they were rounded to (771, where one sum serves the log-sum-exp and the division 729; 300 rows over four
// of 32768 154 with one part and one sum, 163 so, 179 with two parts).
// Both K and V lie in shared memory as the cache holds them, tokens by channels: K is read along its rows,
// V across them.
//
// Roles: a copy warp goes through the CTA's range, describes each segment (a run of an item's pages) to the
// others and fetches queries and pages (TMA), running on into the next segment while this one ends; for each
// tile one warp issues the products for S, as far ahead as S has places, and one those with V; four warps a tile do
// its softmax, a row a thread; one warp looks through V where rows see different tokens: a token that some
// row does not see may hold an infinity or a NaN, which a probability of 0 would not silence, so it is
// zeroed and the rows that do see it are marked.
//
// What bounds it. One tile: memory. A page is 32 KB and takes 0.73 us an SM at the copy rate; the softmax warps
// are busy for less than that. Four sequences of 131072 tokens, 4 heads, 112 rows: 172 to 174 us in a graph,
// 6.2 TB/s, of which the first page's way into the CTA (4 us: lengths, tables, copies, each waiting for the one
// before) and the join (5 to 7) are most of what the floor of 158 lacks. Two tiles: the way round from P to the
// next but one S of a tile. 2048 query tokens over 32768, 32/8 heads, take 765 to 792 us in a graph, 1.37 PFLOP/s or
// 71 % of the measured matrix rate. Clock counts with one sum of the probabilities, 1600 cycles a page: 1270 in a
// row's softmax (the special-function unit's share for two warps a scheduler is 720), 640 of matrix instructions for
// each tile, whose queue both tiles share; the second sum adds about 90, and two parts 256 to each tile's instructions.
// A third place for S would take the way apart; O of two tiles and their four places fill tensor memory,
// and with P in shared memory, which frees S's place sooner, writing it and P V take longer than that saves (716 ->
// 907 us with one part and one sum, with Q in tensor memory in turn 920).
// A short call's time is that of instructions that run once: about 25 cycles each, so set-up is kept short,
// and by a few warps. 4096 tokens, 2 heads, three pages a CTA: 13.2 us in a graph, of them 3.4 to the first
// scores, 2 of pages, 1 of records written, 2 until all others are seen, 2 of copying and 1.5 of joining them.
#include "kv4_walk.cuh"
#include "splitkv.cuh"
#include "tree.cuh"

namespace ffd {
namespace tree {
namespace {

using kv4::Bf16;
using kv4::F16;
using kv4::is_far;
using kv4::kLazy;
using kv4::kMaxCtas;
using kv4::kShift;
using kv4::lse_of;

constexpr int kTile = 128;       // rows of a tile
constexpr int kPageBytes = kPage * kD * 2;
constexpr int kInfo = 8;         // steps whose pages are kept: copies run at most seven ahead of any reader
constexpr int kSegs = 8;         // segments that are kept; each is a step or more
constexpr int kMaskStep = 512;   // blocks whose mask a warp looks at together
constexpr int kMaxUnits = 256;   // (sequence, KV head) pairs whose kept blocks are counted
// Pages' time that a second segment costs a CTA. us with 0 and 4: 60 nodes of 8 heads over 4096 23.3 19.7, 8 nodes of 11
// heads over 16384 28.4 27.6, others the same.
constexpr int kStartPages = 4;
constexpr int kSlots = 2;        // records of a CTA: of the item that goes on from before, and that goes on
constexpr uint32_t kColO = 256;  // O of tile g at kColO + 128 g

template <class T>
struct Idesc {  // instruction words
    static constexpr uint32_t kType = 0;
};
template <>
struct Idesc<Bf16> {
    static constexpr uint32_t kType = kTcBf16;
};

template <int kTiles>
struct Shape {
    static constexpr int kRows = kTile * kTiles;
    static constexpr int kSoft = 4 * kTiles;                 // softmax warps; then
    static constexpr int kCopy = kSoft, kScores = kCopy + 1; // copies, an issuer of S a tile,
    static constexpr int kValues = kScores + kTiles;         // an issuer of P V a tile,
    static constexpr int kClean = kValues + kTiles;          // V's infinities
    static constexpr int kThreads = 32 * (kClean + 1);
    static constexpr int kNK = kTiles == 1 ? 5 : 4;          // pages' K in shared memory
    static constexpr int kNV = kTiles == 1 ? 6 : 5;          // pages' V
    static constexpr int kPlaces = 2;                        // places of S in tensor memory, in turn
    static constexpr int kRecord = 130 * kRows;              // floats of a record: o[128][row], m[row], l[row]
    // tensor memory columns of S (P over its first half)
    static __device__ __forceinline__ uint32_t col_s(int g, uint32_t step) {
        return 64 * (kPlaces * g + step % kPlaces);
    }
};

struct Step {
    int j;     // the page's block index, -1: the segment's end
    int edge;  // some row does not see all of it
};

struct Segment {  // pages 0: there is none any more
    int pages, end;        // how many, and the token behind the last
    int h, t0, nq, first;  // KV head, first node's row, nodes, tokens before the tree
    int node0;             // the item's first node
    int begins, complete;  // whether the segment holds the item's first page, and all of them
    int p0, p1, j0;        // CTAs that share the item, the first that joins it (known at the segment's end)
};

template <int kTiles>
struct Shared {
    using H = Shape<kTiles>;
    uint8_t q[kTiles][2 * 16384];               // tile: channels 0-63, then 64-127
    uint8_t k[H::kNK][kPageBytes];              // the same for a page's tokens
    uint8_t v[H::kNV][kPageBytes];
    uint32_t bits[kMaxNodes / 32][H::kRows];    // nodes that a row sees
    int parent[kTiles][kMaxNodes];
    // barriers, by the number of arrivals: one, kTiles, four
    uint64_t seg_full[kSegs], k_full[H::kNK], v_full[H::kNV], v_ready[H::kNV], q_full, joined;
    uint64_t s_full[kTiles][H::kPlaces], o_done[kTiles][H::kPlaces], drain[2 * kTiles];
    uint64_t k_free[H::kNK], v_free[H::kNV], q_free;
    uint64_t p_full[kTiles][H::kPlaces], end_of_barriers;
    uint64_t bad[H::kNV];                       // tokens of a page whose V is not finite
    Step info[kInfo];
    Segment seg[kSegs];
    uint32_t tmem, aborted;
    int scan[H::kThreads / 32];
    int pre[H::kThreads];                       // weight of all items before each chunk of sequences
    uint16_t list[kMaskStep];                   // kept blocks, counted from a step's first
    int kept[kMaxUnits];                        // blocks that a unit's item has, at least one (0: no item)
    Segment shared_item;                        // the item that this CTA joins (pages 0: none)
};

struct Params {
    CUtensorMap tm_q, tm_k, tm_v;
    AttnArgs a;
    float *records;
    int *tickets;
};

// x / G for a row x of a tile.
__device__ __forceinline__ int div_g(const AttnArgs &a, int x) {
    return a.G == 1 ? x : (int)__umulhi((uint32_t)x, a.over_g);
}

struct Seq {
    int n, t0, nq;  // tokens, first node's row, nodes
    __device__ __forceinline__ int first() const { return n - nq; }  // tokens before the tree
};

__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b, bool report) {
    Seq s;
    s.n = __ldg(a.seq_lens + b);
    s.t0 = b * a.max_q;
    s.nq = a.max_q;
    bool bad = false;
    if (a.cu_q) {
        s.t0 = __ldg(a.cu_q + b);
        const int end = __ldg(a.cu_q + b + 1);
        bad = s.t0 < 0 || end < s.t0 || end > a.total_q || end - s.t0 > a.max_q;
        s.nq = bad ? 0 : end - s.t0;
    }
    const int cap = a.max_blocks * kPage;
    if (s.n > cap) bad = true, s.n = cap;
    if (s.n < s.nq) bad = true, s.n = 0;  // its rows see nothing
    if (report && bad) raise_error(a.err, FFD_ERRBIT_BOUNDS);
    return s;
}

__device__ __forceinline__ int item_groups(const AttnArgs &a, const Seq &s) {
    return s.nq <= a.item_nodes ? s.nq > 0 : (s.nq + a.item_nodes - 1) / a.item_nodes;
}

// Positions of an item's rows: at least lo, at most hi. A node's position is not known here; its
// index bounds its depth.
__device__ __forceinline__ void item_span(const AttnArgs &a, const Seq &s, int rt, int &lo, int &hi) {
    const int i0 = rt * a.item_nodes, i1 = i0 + a.item_nodes;
    lo = s.first() + (a.parents ? 0 : i0);
    hi = s.first() + (i1 < s.nq ? i1 : s.nq) - 1;
}

// Pages that the rows of item group rt of a sequence see: the first, and how many.
__device__ __forceinline__ void item_pages(const AttnArgs &a, const Seq &s, int rt, int &fp, int &np) {
    int lo, hi;
    item_span(a, s, rt, lo, hi);
    fp = a.window > 0 && lo >= a.window ? (lo - a.window + 1) >> 6 : 0;
    np = hi < 0 ? 0 : (hi >> 6) - fp + 1;
}

// What one item weighs, 0 behind the last one: kItemPages before its first page and one for each.
__device__ __forceinline__ int item_weight(const AttnArgs &a, const Seq &s, int rt, int groups) {
    if (rt >= groups) return 0;
    int fp, np;
    item_pages(a, s, rt, fp, np);
    return np > 0 ? np + kItemPages : 0;
}
__device__ __forceinline__ int items_weight(const AttnArgs &a, const Seq &s) {  // of one head
    const int groups = item_groups(a, s);
    int w = 0;
#pragma unroll 1
    for (int rt = 0; rt < groups; rt++) w += item_weight(a, s, rt, groups);
    return w;
}

__device__ __forceinline__ int lane_scan(int v, int lane) {  // sum over the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// One head's items of a sequence, weighed by a warp.
__device__ __forceinline__ int head_weight(const AttnArgs &a, const Seq &s, int lane) {
    int sum = 0;
    const int groups = item_groups(a, s);
    for (int rt = 0; rt < groups; rt += 32) sum += item_weight(a, s, rt + lane, groups);
    return __reduce_add_sync(0xffffffffu, sum);
}

// A word's bytes that are not 0 as their top bits.
__device__ __forceinline__ uint32_t kept_bytes(uint32_t w) {
    return (w | ((w & 0x7f7f7f7fu) + 0x7f7f7f7fu)) & 0x80808080u;
}
__device__ __forceinline__ int chunk_count(const uint4 &x) {
    return __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w);
}
// The mask's bytes at .. at + 15 behind `base` (aligned to 16), 0 outside [lo, hi), by their top bits.
__device__ __forceinline__ uint4 mask_chunk(const uint8_t *base, int at, int lo, int hi) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (at >= lo && at + 16 <= hi) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(base + at));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
#pragma unroll 1
        for (int k = at > lo ? at : lo; k < at + 16 && k < hi; k++) {
            const uint32_t v = __ldg(base + k) ? 1u << (8 * (k & 3)) : 0u;
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] |= (k - at) >> 2 == i ? v : 0u;
        }
    }
    return make_uint4(kept_bytes(w[0]), kept_bytes(w[1]), kept_bytes(w[2]), kept_bytes(w[3]));
}
// How many of n blocks from `mask` on are kept: the share of one of `lanes` threads.
__device__ __forceinline__ int count_kept(const uint8_t *mask, int n, int lane, int lanes) {
    const int before = (int)(-reinterpret_cast<uintptr_t>(mask) & 15);  // bytes before the first 16 aligned ones
    const int head = before < n ? before : n, chunks = (n - head) >> 4, ends = n - 16 * chunks;
    int count = 0;
#pragma unroll 1
    for (int k = lane; k < chunks; k += lanes) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(mask + head) + k);
        count += chunk_count(make_uint4(kept_bytes(x.x), kept_bytes(x.y), kept_bytes(x.z), kept_bytes(x.w)));
    }
    for (int k = lane; k < ends; k += lanes) count += __ldg(mask + (k < head ? k : k + 16 * chunks)) != 0;
    return count;
}
// Output of a sequence's rows that see nothing, a share of them for each CTA.
__device__ __noinline__ void write_empty(const AttnArgs &a, int t0, int nq, int thread, int threads) {
    const int64_t rows = (int64_t)nq * a.Hq, first = (int64_t)t0 * a.Hq;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        for (int c = thread; c < kD / 8; c += threads)
            reinterpret_cast<uint4 *>(a.out + (first + r) * kD)[c] = make_uint4(0, 0, 0, 0);
        if (a.lse && thread == 0) a.lse[first + r] = -INFINITY;
    }
}

// Rows that a channel has in a record of an item that is `left` nodes from its sequence's end: both tiles'
// places up to the last row, in 16 bytes.
__device__ __forceinline__ int record_rows(const AttnArgs &a, int left) {
    const int more = left - a.tile_nodes;
    const int used = more <= 0 || a.item_nodes == a.tile_nodes
                         ? min(left, a.tile_nodes) * a.G : kTile + min(more, a.tile_nodes) * a.G;
    return (used + 3) & ~3;
}

// The weights cut into ncta ranges, the first `more` of them longer by one.
struct Ranges {
    int each, more;
    __device__ __forceinline__ int begin(int cta) const { return cta * each + (cta < more ? cta : more); }
    __device__ __forceinline__ int owner(int x) const {  // the CTA whose range holds x
        const int split = more * (each + 1);
        return x < split ? x / (each + 1) : more + (x - split) / each;
    }
};

// Bounded waits: once one runs out the CTA stops (aborted) and drains what is in flight.
template <class S>
__device__ __forceinline__ bool stopped(const S &sh) {
    return *reinterpret_cast<const volatile uint32_t *>(&sh.aborted) != 0;
}
template <class S>
__device__ __noinline__ bool wait_long(const AttnArgs &a, S &sh, uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (stopped(sh)) return false;
        if (globaltimer_ns() - t0 > a.wait_ns) {
            raise_error(a.err, FFD_ERRBIT_TIMEOUT);
            *reinterpret_cast<volatile uint32_t *>(&sh.aborted) = 1;
            return false;
        }
    }
    return true;
}
// By a whole warp: true once the phase is complete, false when the CTA has stopped.
template <class S>
__device__ __forceinline__ bool waited(const AttnArgs &a, S &sh, uint64_t *bar, uint32_t parity) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_long(a, sh, bar, parity);
    return __all_sync(0xffffffffu, ok);
}

// Bits 0 .. k of a word (none below 0, all from 63 on).
__device__ __forceinline__ uint64_t upto(int k) {
    return k < 0 ? 0ull : k >= 63 ? ~0ull : (2ull << k) - 1;
}

template <class T, int kTiles, int kParts>
__global__ void __launch_bounds__(Shape<kTiles>::kThreads, 1)
    tree_kernel(const __grid_constant__ Params prm) {
    using H = Shape<kTiles>;
    constexpr int kRows = H::kRows, kThreads = H::kThreads, kCtaWarps = kThreads / 32;
    constexpr int kPlaces = H::kPlaces;
    static_assert(H::kNV + 1 < kInfo && H::kNV + 1 < kSegs, "what copies run ahead");
    extern __shared__ uint8_t raw[];
    using Sh = Shared<kTiles>;
    Sh &sh = *reinterpret_cast<Sh *>(align_shared<1024>(raw));
    static_assert(sizeof(Sh) + 1024 <= 232448, "shared memory per CTA");
    const AttnArgs &a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // Tables set out for L2 while the lengths are read, by warps that are idle yet (96 kept blocks of 4 x 131072,
    // 25 nodes: 0.6 of 31 us, 64 of 32 x 30000 to 131072, 8 nodes of 4 heads: 2 of 68).
    if (warp < H::kSoft) {
        const int64_t at = 128 * ((int64_t)blockIdx.x * kRows + tid), entries = (int64_t)a.B * a.max_blocks;
        if (at < 4 * entries) prefetch_l2(reinterpret_cast<const uint8_t *>(a.block_table) + at);
        if (a.by_mask && at < entries * a.Hkv) prefetch_l2(a.keep_in + at);
    }
    __syncwarp();
    if (warp == 0) tmem_alloc(&sh.tmem, 512);
    if (warp == 1) {
        uint64_t *one = sh.seg_full, *tiles = sh.k_free, *four = sh.p_full[0], *end = &sh.end_of_barriers;
        for (uint64_t *bar = one + lane; bar < end; bar += 32)
            mbar_init(bar, bar >= four ? 4 : bar >= tiles ? kTiles : 1);
        if (lane == 0) sh.aborted = 0, sh.shared_item.pages = 0;
        fence_barrier_init();
    }
    // ---- weight of all items: up to 32 sequences by the copy warp alone, a lane each; more by all threads, a
    // run of sequences each
    const bool few = a.B <= 32;
    const int chunk = (a.B + kThreads - 1) / kThreads;  // sequences of a thread
    int total = 0, own = 0;
    Seq s = {0, 0, 0};
    if (few) {
        // by all threads, 4 to 32 a unit; each CTA begins elsewhere, so that not all ask for the same bytes
        if (a.by_mask) {
            const int units = a.B * a.Hkv;
            int log = 5;
            while (log > 2 && units << log > kThreads) log--;
            const int shift = (int)blockIdx.x * units / (int)gridDim.x;
#pragma unroll 1
            for (int u0 = 0; u0 < units; u0 += kThreads >> log) {
                int u = u0 + (tid >> log);
                if (u < units && (u += shift) >= units) u -= units;
                const int part = tid & ((1 << log) - 1);
                int fp = 0, np = 0, kept = 0;
                if (u < units) {
                    const Seq e = seq_of(a, u / a.Hkv, false);
                    if (e.nq > 0) item_pages(a, e, 0, fp, np);
                    kept = count_kept(a.keep_in + (int64_t)u * a.max_blocks + fp, np, part, 1 << log);
                }
                for (int o = 1 << log >> 1; o; o >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, o);
                if (u < units && part == 0) sh.kept[u] = np > 0 ? max(kept, 1) : 0;
            }
        }
        if (warp == H::kCopy) {
            if (lane < a.B) {
                s = seq_of(a, lane, blockIdx.x == 0);
                own = items_weight(a, s) * a.Hkv;
            }
        } else if (warp == H::kClean) {
            Seq e = {1, 0, 0};
            if (lane < a.B) e = seq_of(a, lane, false);
            for (uint32_t todo = __ballot_sync(0xffffffffu, e.n == 0 && e.nq > 0); todo; todo &= todo - 1) {
                const int b = __ffs(todo) - 1;
                write_empty(a, __shfl_sync(0xffffffffu, e.t0, b), __shfl_sync(0xffffffffu, e.nq, b), lane, 32);
            }
        }
    } else {
        bool empty = false;  // some sequence's rows see nothing
#pragma unroll 1
        for (int b = tid * chunk; b < (tid + 1) * chunk && b < a.B; b++) {
            const Seq e = seq_of(a, b, blockIdx.x == 0);
            own += items_weight(a, e) * a.Hkv;
            empty |= e.n == 0 && e.nq > 0;
        }
        empty = __syncthreads_or(empty);
        const int inc = lane_scan(own, lane);
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        const int of_warp = lane_scan(lane < kCtaWarps ? sh.scan[lane] : 0, lane);
        total = __shfl_sync(0xffffffffu, of_warp, 31);
        const int warps = __shfl_sync(0xffffffffu, of_warp, warp == 0 ? 0 : warp - 1);
        sh.pre[tid] = (warp == 0 ? 0 : warps) + inc - own;
        if (empty) {
#pragma unroll 1
            for (int b = 0; b < a.B; b++) {
                const Seq e = seq_of(a, b, false);
                if (e.n == 0) write_empty(a, e.t0, e.nq, tid, kThreads);
            }
        }
    }
    const int cta = blockIdx.x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    uint32_t steps = 0, segs = 0;  // so far; a segment's end is a step too
    bool issuer = false;  // the lane that issues a warp's matrix instructions
    uint32_t keys = 0;    // 1 when the copy warp stopped between a page's K and V
    // The next segment's description; null at the range's end or when the CTA has stopped.
    auto next_segment = [&]() -> const Segment * {
        const uint32_t at = segs % kSegs, parity = (segs / kSegs) & 1;
        segs++;
        if (!waited(a, sh, &sh.seg_full[at], parity)) return nullptr;
        return sh.seg[at].pages > 0 ? &sh.seg[at] : nullptr;
    };
    if (warp < H::kSoft) {
        // ================= softmax of tile grp, one row a thread =================
        const int grp = warp >> 2, r = tid & (kTile - 1);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t to = tmem + lanes + kColO + grp * 128;
        const int rn = div_g(a, r), rg = r - rn * a.G;  // the row's node in the tile, and head
        const float fs = a.factor;
        while (true) {
            const Segment *sg = next_segment();
            if (named_barrier_or(3, kRows, sg == nullptr)) break;
            const int first = sg->first, nq = sg->nq, node0 = sg->node0, t0 = sg->t0;
            const bool active = grp == 0 || nq - node0 > a.tile_nodes;
            const bool complete = sg->complete;
            const int qi = node0 + grp * a.tile_nodes + rn;
            const bool have = rn < a.tile_nodes && qi < nq;
            // ---- the nodes that the row sees, and its position
            int pos = first + qi;
            if (a.parents && (sg->end > first || a.window > 0)) {
                for (int i = r; i < nq; i += kTile) {
                    int p = __ldg(a.parents + t0 + i);
                    if (p < -1 || p >= i) {
                        raise_error(a.err, FFD_ERRBIT_BOUNDS);
                        p = -1;
                    }
                    sh.parent[grp][i] = p;
                }
                named_barrier_sync(1 + grp, kTile);
                uint32_t bits[kMaxNodes / 32] = {};
                int depth = 0;
                if (have) {
                    for (int x = qi;; depth++) {
                        if (a.window == 0 || depth < a.window) {
#pragma unroll
                            for (int k = 0; k < kMaxNodes / 32; k++)
                                bits[k] |= (x >> 5) == k ? 1u << (x & 31) : 0u;
                        }
                        x = sh.parent[grp][x];
                        if (x < 0) break;
                    }
                }
                pos = first + depth;
#pragma unroll
                for (int k = 0; k < kMaxNodes / 32; k++) sh.bits[k][grp * kTile + r] = bits[k];
                named_barrier_sync(1 + grp, kTile);  // the parents have been read
            }
            const int from = a.window > 0 ? pos - a.window : -1;
            // Tokens of page j that the row sees.
            auto visible = [&](int j) -> uint64_t {
                const int t = 64 * j;
                if (!a.parents) return upto(pos - t) & ~upto(from - t);
                uint64_t see = upto(first - 1 - t) & ~upto(from - t);
                const int x = t - first;  // the page's first token as a node
                if (x + 63 >= 0) {
                    // nodes x .. x + 63: three words
                    const int k = x >> 5;
                    auto word = [&](int i) {
                        return i >= 0 && i < kMaxNodes / 32 ? sh.bits[i][grp * kTile + r] : 0u;
                    };
                    const uint32_t w0 = word(k), w1 = word(k + 1), w2 = word(k + 2);
                    see |= (uint64_t)__funnelshift_r(w1, w2, x & 31) << 32 | __funnelshift_r(w0, w1, x & 31);
                }
                return have ? see : 0ull;
            };

            float m = -INFINITY, limit = -INFINITY, l = 0.0f;  // limit: a larger score raises m
            float lr = 0.0f;  // what l is of the rounded probabilities, where they have one part
            bool any = false, far = false, tainted = false;
            while (true) {
                const uint32_t buf = steps % kPlaces, vs = steps % H::kNV;
                if (!waited(a, sh, &sh.s_full[grp][buf], (steps / kPlaces) & 1)) break;
                tc_fence_after();
                const volatile Step &info = sh.info[steps % kInfo];
                const int j = info.j, edge = info.edge;
                const uint32_t ts = tmem + lanes + H::col_s(grp, steps);
                if (j >= 0 && active) {
                    const uint64_t see = edge ? visible(j) : ~0ull;
                    uint32_t x[64];
                    __syncwarp();
                    tmem_load32(reinterpret_cast<uint32_t(&)[32]>(x[0]), ts);
                    tmem_load32(reinterpret_cast<uint32_t(&)[32]>(x[32]), ts + 32);
                    tc_wait_load();
                    if (edge) {
                        const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
                        for (int c = 0; c < 32; c++) {
                            if (!((lo >> c) & 1u)) x[c] = 0xff800000u;
                            if (!((hi >> c) & 1u)) x[32 + c] = 0xff800000u;
                        }
                    }
                    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            t[e] = fmaxf(t[e], fmaxf(__uint_as_float(x[c + 2 * e]),
                                                     __uint_as_float(x[c + 2 * e + 1])));
                    const float top = fs * fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                    const bool raise = have && top > limit;  // (a tile's spare rows hold anything)
                    if (__any_sync(0xffffffffu, raise)) {
                        const float mn = raise ? top : m;
                        const float al = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
                        m = mn;
                        limit = m + (is_far(m) ? 0.0f : kLazy);
                        l *= al;
                        lr *= al;
                        far = __any_sync(0xffffffffu, is_far(m));
                        if (any) {
                            // the last step's P V (a stop is met at the next wait)
                            waited(a, sh, &sh.o_done[grp][(steps - 1) % kPlaces], ((steps - 1) / kPlaces) & 1);
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < 4; c++) {
                                uint32_t o[32];
                                tmem_load32(o, to + 32 * c);
                                tc_wait_load();
#pragma unroll
                                for (int e = 0; e < 32; e++)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                tmem_store32(to + 32 * c, o);
                            }
                            tc_wait_store();
                        }
                    }
                    const float sub = kShift - (m == -INFINITY ? 0.0f : m);
                    const float fx = far ? 1.0f : fs;
                    const float2 f2 = make_float2(fx, fx), s2 = make_float2(sub, sub);
                    float2 l2 = make_float2(0.0f, 0.0f), l3 = l2;
                    if (far) {
#pragma unroll
                        for (int c = 0; c < 64; c++)
                            x[c] = __float_as_uint(__fmul_rn(__uint_as_float(x[c]), fs));
                    }
                    float2 r2 = l2, r3 = l2;
                    uint32_t p[kParts][32];  // as numbers of T: rounded, and the rest
#pragma unroll
                    for (int c = 0; c < 32; c++) {
                        float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]),
                                                          __uint_as_float(x[2 * c + 1])), f2, s2);
                        e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                        if (c & 1) l3 = __fadd2_rn(l3, e);
                        else l2 = __fadd2_rn(l2, e);
                        p[0][c] = T::pack(e.x, e.y);
                        const float2 first = T::unpack(p[0][c]);
                        if constexpr (kParts == 2) {
                            const float2 rest = __ffma2_rn(first, make_float2(-1.0f, -1.0f), e);
                            p[1][c] = T::pack(rest.x, rest.y);
                        } else {
                            if (c & 1) r3 = __fadd2_rn(r3, first);
                            else r2 = __fadd2_rn(r2, first);
                        }
                    }
                    __syncwarp();
                    // 32 columns a part, over S's, which have been read
#pragma unroll
                    for (int i = 0; i < kParts; i++) tmem_store32(ts + 32 * i, p[i]);
                    l += (l2.x + l2.y) + (l3.x + l3.y);
                    if (kParts == 1) lr += (r2.x + r2.y) + (r3.x + r3.y);
                    if (edge && waited(a, sh, &sh.v_ready[vs], (steps / H::kNV) & 1))
                        tainted |= (*reinterpret_cast<volatile uint64_t *>(&sh.bad[vs]) & see) != 0;
                    tc_wait_store();
                    any = true;
                }
                steps++;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[grp][buf]);  // at a segment's end too
                if (j < 0) break;
            }
            if (any) {  // the last page's P V: two steps back, behind it the end
                waited(a, sh, &sh.o_done[grp][(steps - 2) % kPlaces], ((steps - 2) / kPlaces) & 1);
                tc_fence_after();
            }
            if (named_barrier_or(3, kRows, stopped(sh))) break;

            // ---- the segment's results
            const int begins = sg->begins;
            if (active) {
                // O by the weights that it was summed with
                const float even = kParts == 1 && lr > 0.0f ? l / lr : 1.0f;
                const float inv = tainted ? NAN : l == 0.0f ? 0.0f : even / l;
                const int pad = record_rows(a, nq - node0);
                float *row = prm.records + (int64_t)(kSlots * cta + begins) * H::kRecord + grp * kTile + r;
                const int64_t at = (int64_t)(t0 + qi) * a.Hq + sg->h * a.G + rg;
#pragma unroll 1
                for (int c = 0; c < 4; c++) {
                    uint32_t o[32];
                    __syncwarp();
                    if (any) {  // warp-uniform
                        tmem_load32(o, to + 32 * c);
                        tc_wait_load();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e++) o[e] = 0;
                    }
                    if (!have) continue;
                    if (complete) {
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 8; k++)
                                y[k] = T::pack(__uint_as_float(o[16 * e + 2 * k]) * inv,
                                               __uint_as_float(o[16 * e + 2 * k + 1]) * inv);
                            uint16_t *dst = a.out + at * kD + 32 * c + 16 * e;
                            if (a.wide_out) {
                                store_32b(dst, y);
                            } else {
                                reinterpret_cast<uint4 *>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                                reinterpret_cast<uint4 *>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            row[(32 * c + e) * pad] = tainted ? NAN : __uint_as_float(o[e]) * even;
                    }
                }
                if (have) {
                    if (!complete) row[128 * pad] = m, row[129 * pad] = l;
                    else if (a.lse) a.lse[at] = lse_of(m - kShift, l);
                }
            }
            if (!complete) {  // joined below
                fence_proxy_async_all();  // the records are read by bulk copies
                if (tid == 0 && cta >= sg->j0) sh.shared_item = *sg;
                named_barrier_sync(3, kRows);
                if (tid == 0) add_acq_rel_gpu(prm.tickets + sg->p0, 1);
            }
        }
        // ---- the shared item: it began before this CTA's range, or each CTA has a share of one item
        if (!named_barrier_or(3, kRows, stopped(sh)) && sh.shared_item.pages > 0) {
            const Segment &c = sh.shared_item;
            const int n = c.p1 - c.p0 + 1, place = cta - c.j0, of = c.p1 - c.j0 + 1;
            // channels by eights, of many CTAs by twos: at most eight of them then
            const int unit = of <= 16 ? 8 : 2, units = kD / unit;
            const int ch0 = units * place / of * unit, chs = units * (place + 1) / of * unit - ch0;
            const int pad = record_rows(a, c.nq - c.node0);
            float *buf = reinterpret_cast<float *>(sh.q[0]);
            constexpr int kRoom = (sizeof(sh.q) + sizeof(sh.k) + sizeof(sh.v)) / 4;
            // Channels that are joined together: as many of this CTA's as have room with all records, in
            // eights; eight at least, in several rounds of records where need be.
            const int most = (kRoom / (n * pad) - 2) & ~7;
            const int block = min(chs, most < 8 ? 8 : most);
            const int once = min(n, kRoom / ((block + 2) * pad));
            if (tid == 0) {
                const uint64_t t0 = globaltimer_ns();
                bool ok = true;
                while (ok && ld_acquire_gpu(prm.tickets + c.p0) < n) ok = globaltimer_ns() - t0 <= a.wait_ns;
                if (!ok) {
                    raise_error(a.err, FFD_ERRBIT_TIMEOUT);
                    *reinterpret_cast<volatile uint32_t *>(&sh.aborted) = 1;
                } else if (atomicAdd(prm.tickets + kMaxCtas + c.p0, 1) == of - 1) {
                    // nobody waits any more: both counters are left at 0 for the next call
                    prm.tickets[c.p0] = prm.tickets[kMaxCtas + c.p0] = 0;
                }
            }
            const bool run = !named_barrier_or(3, kRows, stopped(sh));
            uint32_t rounds = 0;
            // A thread takes a row and eight channels at a time, rows along the threads. Several rounds of
            // records come where there are eight channels at most, and no more units than threads.
            float M = -INFINITY, ls = 0.0f, o[8];
#pragma unroll 1
            for (int b0 = 0; run && b0 < chs; b0 += block) {
                const int width = min(block, chs - b0), rec = (width + 2) * pad;  // rec: a record's floats
#pragma unroll 1
                for (int r0 = 0; r0 < n; r0 += once) {
                    const int count = min(once, n - r0);
                    fence_proxy_async_all();
                    if (tid == 0) mbar_arrive_expect_tx(&sh.joined, count * rec * 4);
                    named_barrier_sync(3, kRows);  // the space has been read
                    for (int k = tid; k < count; k += kRows) {  // a record each
                        const int p = r0 + k;
                        const float *src =  // a CTA's second record where the item begins, else its first
                            prm.records + (int64_t)(kSlots * (c.p0 + p) + (p == 0)) * H::kRecord;
                        tma_load_1d(buf + k * rec, src + (ch0 + b0) * pad, width * pad * 4, &sh.joined);
                        tma_load_1d(buf + k * rec + width * pad, src + kD * pad, 2 * pad * 4, &sh.joined);
                    }
                    if (!mbar_drain(&sh.joined, rounds & 1, drain_bound_ns(a.wait_ns)))
                        raise_error(a.err, FFD_ERRBIT_TIMEOUT);
                    rounds++;
                    int x0 = 0, q = tid;  // the unit's first channel and row
                    while (q >= pad) q -= pad, x0 += 8;
#pragma unroll 1
                    while (x0 < width) {
                        const float *mine = buf + x0 * pad + q, *ms = buf + width * pad + q;
                        if (r0 == 0) {
                            M = -INFINITY, ls = 0.0f;
#pragma unroll
                            for (int x = 0; x < 8; x++) o[x] = 0.0f;
                        }
                        float Mn = M;
#pragma unroll 8
                        for (int k = 0; k < count; k++) Mn = fmaxf(Mn, ms[k * rec]);
                        if (r0 > 0) {
                            const float al = M == -INFINITY ? 0.0f : ex2_approx(M - Mn);
                            ls *= al;
#pragma unroll
                            for (int x = 0; x < 8; x++) o[x] *= al;
                        }
                        M = Mn;
                        const float ref = M == -INFINITY ? 0.0f : M;  // nothing in any: o and l are 0
#pragma unroll 4
                        for (int k = 0; k < count; k++) {
                            const float f = ex2_approx(ms[k * rec] - ref);
                            ls = fmaf(f, ms[k * rec + pad], ls);
#pragma unroll
                            for (int x = 0; x < 8; x++)
                                if (x0 + x < width) o[x] = fmaf(f, mine[k * rec + x * pad], o[x]);
                        }
                        const int g = q >= kTile, rr = q - g * kTile, node = div_g(a, rr);
                        const int i = c.node0 + g * a.tile_nodes + node;
                        if (r0 + count >= n && node < a.tile_nodes && i < c.nq) {
                            const int64_t at = (int64_t)(c.t0 + i) * a.Hq + c.h * a.G + rr - node * a.G;
                            const int ch = ch0 + b0 + x0;
                            const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                            uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + at * kD + ch);
                            const uint32_t y[4] = {T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv),
                                                   T::pack(o[4] * inv, o[5] * inv), T::pack(o[6] * inv, o[7] * inv)};
                            if (unit == 8) {
                                *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; k++)
                                    if (2 * k < width) dst[k] = y[k];
                            }
                            if (a.lse && ch == 0) a.lse[at] = lse_of(M - kShift, ls);
                        }
                        q += kRows;
                        while (q >= pad) q -= pad, x0 += 8;
                    }
                }
            }
        }
    } else if (warp == H::kCopy) {
        // ================= the range's segments, copies of their queries and pages =================
        if (lane == 0) {
            prefetch_tensormap(&prm.tm_q);
            prefetch_tensormap(&prm.tm_k);
            prefetch_tensormap(&prm.tm_v);
        }
        const int several = a.by_mask ? (a.B * a.Hkv + 31) / 32 : 0;  // units of a lane, where blocks are counted
        int longest = 0;  // pages of the longest of the lane's items
        if (several) {
            own = 0;
            for (int u = several * lane; u < several * (lane + 1) && u < a.B * a.Hkv; u++) {
                own += sh.kept[u] ? sh.kept[u] + kItemPages : 0;
                longest = max(longest, sh.kept[u]);
            }
        }
        const int inc = lane_scan(own, lane);
        if (few) total = __shfl_sync(0xffffffffu, inc, 31);
        int ncta = min(total, (int)gridDim.x), x, c1, b = 0, h = 0, rt = 0, into = 0, per = 0;
        if (a.shares > 0 && total > 0) {
            // No more items than CTAs, of about one length: each in equal shares of `per` pages, so that no CTA has
            // the end of one and the start of another, unless that leaves too many CTAs without work. Measured,
            // us by shares and cut regardless (152 CTAs, before items
            // cut regardless went in shares of share_pages): 8 heads of 32768 tokens, 16 nodes 34 37; of 131072
            // 88 94; one head of 32768, 60 nodes 28 34; ten heads of 8192 19 25.
            const bool full = lane >= a.B || s.nq > (a.groups - 1) * a.item_nodes;  // all its groups are there
            if (!several) {  // (behind a window it need not be the last group's)
#pragma unroll 1
                for (int g = 0; lane < a.B && g < a.groups; g++) {
                    int fp, np;
                    item_pages(a, s, g, fp, np);
                    longest = max(longest, np);
                }
            }
            const int np = __reduce_max_sync(0xffffffffu, longest);
            per = a.over_shares ? (int)__umulhi(np + a.shares - 1, a.over_shares) : np;
            if (!__all_sync(0xffffffffu, full) || (int64_t)(per - kStartPages) * gridDim.x > total) per = 0;
            else per = max(per, share_pages(np));
        }
        const int lead = per ? 0 : kItemPages;
        const Ranges ranges = per ? Ranges{per, 0} : Ranges{total / max(ncta, 1), total % max(ncta, 1)};
        if (per) {  // item by item: groups of a head, heads, sequences
            const int item = a.over_shares ? (int)__umulhi(cta, a.over_shares) : cta;
            const int unit = a.over_groups ? (int)__umulhi(item, a.over_groups) : item;
            b = a.over_heads ? (int)__umulhi(unit, a.over_heads) : unit;
            h = unit - b * a.Hkv;
            rt = item - unit * a.groups;
            into = (cta - item * a.shares) * per;
            x = cta * per;
            c1 = b < a.B ? x + per : x;
            s.n = __shfl_sync(0xffffffffu, s.n, b);
            s.t0 = __shfl_sync(0xffffffffu, s.t0, b);
            s.nq = __shfl_sync(0xffffffffu, s.nq, b);
            ncta = 0;  // found
        } else {
            x = ranges.begin(cta);
            c1 = cta < ncta ? ranges.begin(cta + 1) : x;
        }
        if (cta < ncta) {  // where the range begins: sequence b, head h, group rt, `into` the item's weight
            int rem = x, hp = 1;
            if (few) {
                b = __ffs(__ballot_sync(0xffffffffu, inc > x)) - 1;
                rem -= __shfl_sync(0xffffffffu, inc - own, b);
                if (several) {
                    int u = several * b;
                    for (;; u++) {
                        hp = sh.kept[u] ? sh.kept[u] + kItemPages : 0;
                        if (rem < hp) break;
                        rem -= hp;
                    }
                    b = u / a.Hkv;
                    h = u - b * a.Hkv;
                    hp = 1 << 30;
                } else {
                    hp = __shfl_sync(0xffffffffu, own, b) / a.Hkv;
                }
                s.n = __shfl_sync(0xffffffffu, s.n, b);
                s.t0 = __shfl_sync(0xffffffffu, s.t0, b);
                s.nq = __shfl_sync(0xffffffffu, s.nq, b);
            } else {
                int lo = 0, hi = kThreads;  // the last chunk of sequences that begins at or before x
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (sh.pre[mid] <= x) lo = mid;
                    else hi = mid;
                }
                rem -= sh.pre[lo];
#pragma unroll 1
                for (b = lo * chunk; b < a.B; b++) {
                    s = seq_of(a, b, false);
                    hp = head_weight(a, s, lane);
                    if (rem < hp * a.Hkv) break;
                    rem -= hp * a.Hkv;
                }
            }
            if (rem >= hp) {
                h = rem / hp;
                rem -= h * hp;
            }
            const int groups = item_groups(a, s);
            if (groups > 1) {
#pragma unroll 1
                for (;; rt += 32) {  // 32 items at a time
                    const int wt = item_weight(a, s, rt + lane, groups);
                    const int sum = lane_scan(wt, lane);
                    const uint32_t past = __ballot_sync(0xffffffffu, sum > rem);
                    if (past) {
                        const int k = __ffs(past) - 1;
                        rem -= __shfl_sync(0xffffffffu, sum - wt, k);
                        rt += k;
                        break;
                    }
                    rem -= __shfl_sync(0xffffffffu, sum, 31);
                }
            }
            into = rem;
        }
        bool fine = true;
        while (fine) {
            int fp = 0, np = 0, len = 0, item = 0, at = 0, cnt = 0;  // item: its first page in the cut's scale
            const uint8_t *keep = a.keep_in ? a.keep_in + ((int64_t)b * a.Hkv + h) * a.max_blocks : nullptr;
            if (x < c1) {
                item_pages(a, s, rt, fp, np);
                len = several ? sh.kept[b * a.Hkv + h] : np;  // pages that are counted
                item = x - into + lead;
                at = into > lead ? into - lead : 0;
                cnt = min(len, c1 - item) - at;  // not above 0: the item's pages are the next CTA's
            }
            const int begin = fp + at, end = several ? fp + np : begin + cnt;
            const int node0 = rt * a.item_nodes;
            const int32_t *bt = a.block_table + (int64_t)b * a.max_blocks;
            auto look = [&](int j) {  // -1: dropped, -2: kept, but out of range
                int p = -1;
                if (j < end) {
                    p = __ldg(bt + j);  // beside the mask: it has the same way to go
                    if (keep && !__ldg(keep + j)) p = -1;
                    else if (p < 0 || p >= a.P) p = -2;
                }
                return p;
            };
            // under way while the segment is described: pages, or the mask of the item's first blocks
            const int lo16 = (int)(reinterpret_cast<uintptr_t>(keep + fp) & 15), past = lo16 + np;
            auto flags_at = [&](int from) { return mask_chunk(keep + fp - lo16, from + 16 * lane, lo16, past); };
            int ahead = -1;
            uint4 flags = make_uint4(0, 0, 0, 0);
            if (cnt > 0 && several) flags = flags_at(0);
            else if (cnt > 0) ahead = look(begin + lane);
            if (lane == 0) {
                Segment &d = sh.seg[segs % kSegs];
                d.pages = cnt > 0 ? cnt : 0;
                if (cnt > 0) {
                    // (five kept blocks behind the segment's: none of its own holds a node)
                    d.end = several && len - (at + cnt) >= (kMaxNodes - 1) / kPage + 2 ? 0 : end * kPage;
                    d.h = h, d.t0 = s.t0, d.nq = s.nq, d.first = s.first(), d.node0 = node0;
                    d.begins = at == 0;
                    d.complete = at == 0 && cnt == len;
                }
                mbar_arrive(&sh.seg_full[segs % kSegs]);
            }
            if (cnt <= 0) break;
            if (segs > 0 && !waited(a, sh, &sh.q_free, (segs - 1) & 1)) break;
            if (lane == 0) {  // rows of tile g: nodes by heads, as a box of {64 channels, G heads, nodes}
                const int tiles = kTiles == 2 && s.nq - node0 > a.tile_nodes ? 2 : 1;
                mbar_arrive_expect_tx(&sh.q_full, tiles * a.tile_nodes * a.G * kD * 2);
                for (int g = 0; g < tiles; g++)
#pragma unroll
                    for (int c = 0; c < 2; c++)
                        tma_load_3d(sh.q[g] + c * 16384, &prm.tm_q, 64 * c, h * a.G,
                                    s.t0 + node0 + g * a.tile_nodes, &sh.q_full);
            }
            segs++;
            int lo, hi;
            item_span(a, s, rt, lo, hi);
            const int seen = a.parents ? lo - 1 : lo;  // tokens up to here are seen by all, but for a window
            const int from = a.window > 0 ? hi - a.window : -1;  // and those behind here
            auto edge = [&](int j) { return 64 * j + 63 > seen || 64 * j <= from; };
            auto push = [&](int j, int p) {  // a page (j < 0: the segment's end)
                const uint32_t ks = steps % H::kNK, vs = steps % H::kNV;
                if (steps >= H::kNK && !waited(a, sh, &sh.k_free[ks], (steps / H::kNK - 1) & 1)) return false;
                if (lane == 0) {
                    volatile Step &info = sh.info[steps % kInfo];
                    info.j = j;
                    info.edge = j >= 0 && edge(j);
                    if (j >= 0) {
                        mbar_arrive_expect_tx(&sh.k_full[ks], kPageBytes);
                        tma_load_3d(sh.k[ks], &prm.tm_k, 0, (p * a.Hkv + h) * kPage, 0, &sh.k_full[ks]);
                    } else {
                        mbar_arrive(&sh.k_full[ks]);
                    }
                }
                if (steps >= H::kNV && !waited(a, sh, &sh.v_free[vs], (steps / H::kNV - 1) & 1)) {
                    keys = 1;
                    return false;
                }
                if (lane == 0) {
                    if (j >= 0) {
                        mbar_arrive_expect_tx(&sh.v_full[vs], kPageBytes);
                        tma_load_3d(sh.v[vs], &prm.tm_v, 0, (p * a.Hkv + h) * kPage, 0, &sh.v_full[vs]);
                    } else {
                        mbar_arrive(&sh.v_full[vs]);
                    }
                }
                steps++;
                return true;
            };
            // Pages a batch of 32 at a time. Counted masks are listed first, so that a few kept blocks of many cost
            // no reads one after another (64 of up to 2048 blocks, 32 sequences, 4 heads: 95 us with batches of 32
            // blocks, 79 so).
            int left = cnt, jb = begin;                        // pages to go (counted masks); the next block (others)
            int next = 0, skip = at, i = 0, all = 0, base = 0;  // counted masks: next step, kept ones to pass, list
            while (fine) {
                int block = 0, page = -1;
                if (several) {
                    while (i >= all && next < past) {
                        const int count = chunk_count(flags), sum = lane_scan(count, lane);
                        all = __shfl_sync(0xffffffffu, sum, 31);
                        if (skip < all) {
                            __syncwarp();  // the list has been read
                            int n = sum - count;
                            const uint32_t w[4] = {flags.x, flags.y, flags.z, flags.w};
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                for (uint32_t v = w[q]; v; v &= v - 1)
                                    sh.list[n++] = 16 * lane + 4 * q + ((__ffs(v) - 1) >> 3);
                            __syncwarp();
                            i = skip;
                            skip = 0;
                            base = fp + next - lo16;
                        } else {
                            skip -= all;
                            i = all = 0;
                        }
                        next += kMaskStep;
                        if (next < past) flags = flags_at(next);
                    }
                    const int n = min(32, min(all - i, left));
                    if (n <= 0) break;
                    if (lane < n) {
                        block = base + sh.list[i + lane];
                        page = __ldg(bt + block);
                        if (page < 0 || page >= a.P) page = -2;
                    }
                    i += 32;
                    left -= n;
                } else {
                    if (jb >= end) break;
                    block = jb + lane;
                    page = ahead;
                    jb += 32;
                    ahead = look(jb + lane);
                }
                for (uint32_t todo = __ballot_sync(0xffffffffu, page != -1); todo && fine; todo &= todo - 1) {
                    const int k = __ffs(todo) - 1, p = __shfl_sync(0xffffffffu, page, k);
                    const int j = __shfl_sync(0xffffffffu, block, k);
                    if (p >= 0) fine = push(j, p);
                    else if (lane == 0) raise_error(a.err, FFD_ERRBIT_BOUNDS);
                }
            }
            if (lane == 0) {  // before the end is told of
                Segment &d = sh.seg[(segs - 1) % kSegs];
                d.p0 = ranges.owner(item), d.p1 = ranges.owner(item + len - 1), d.j0 = d.p0 + (per == 0);
            }
            fine = fine && push(-1, 0);
            // ---- the next item that has pages
            x = per ? c1 : item + at + cnt;
            into = 0;
            if (x >= c1) continue;
            do {
                if (++rt >= item_groups(a, s)) {
                    rt = 0;
                    if (++h >= a.Hkv) {
                        h = 0;
                        do s = seq_of(a, ++b, false);
                        while (s.nq == 0);
                    }
                }
                item_pages(a, s, rt, fp, np);
            } while (np == 0);  // (an item with pages counts for one block at least)
        }
    } else if (warp < H::kClean) {
        // ================= matrix instructions of one tile =================
        // The whole warp goes through the steps, so that operand addresses stay warp-uniform; one lane
        // issues.
        issuer = elect_one();
        const bool scores = warp < H::kValues;
        const int g = warp - (scores ? H::kScores : H::kValues);
        if (scores) {
            const uint32_t k0 = smem_u32(sh.k[0]), qd = tc_desc(smem_u32(sh.q[g]));
            bool fine = true;
            while (fine) {
                const Segment *sg = next_segment();
                if (!sg) break;
                const bool live = g == 0 || sg->nq - sg->node0 > a.tile_nodes;
                fine = waited(a, sh, &sh.q_full, (segs - 1) & 1);
                while (fine) {
                    const uint32_t ks = steps % H::kNK, buf = steps % kPlaces, d = tmem + H::col_s(g, steps);
                    if (!(fine = waited(a, sh, &sh.k_full[ks], (steps / H::kNK) & 1))) break;
                    const volatile Step &info = sh.info[steps % kInfo];
                    const bool page = __shfl_sync(0xffffffffu, info.j, 0) >= 0;
                    const uint32_t kd = tc_desc(k0 + ks * kPageBytes);
                    // The place's last P has been taken in (an end: been seen), and its S before. What a tile
                    // goes round by: nothing is left to do behind it (2048 tokens over 32768, 32/8 heads:
                    // 771 us with K waited for behind it, 735 so).
                    if (steps >= kPlaces &&
                        !(fine = waited(a, sh, &sh.o_done[g][buf], (steps / kPlaces - 1) & 1)))
                        break;
                    tc_fence_after();
                    constexpr uint32_t kIdescS = tc_idesc_f16(128, 64) | Idesc<T>::kType;
                    if (issuer) {
                        if (page && live) {
#pragma unroll
                            for (int i = 0; i < 8; i++)  // 16 channels each
                                tc_mma(d, qd + (i >> 2) * 1024 + (i & 3) * 2,
                                       kd + (i >> 2) * 512 + (i & 3) * 2, kIdescS, i > 0);
                        }
                        tc_commit(&sh.s_full[g][buf]);
                        tc_commit(&sh.k_free[ks]);
                        if (!page) tc_commit(&sh.q_free);
                    }
                    steps++;
                    if (!page) break;
                }
            }
        } else {
            const uint32_t v0 = smem_u32(sh.v[0]), d = tmem + kColO + g * 128;
            constexpr uint32_t kIdescO = tc_idesc_f16(128, 128) | Idesc<T>::kType | kTcBMn;
            bool fine = true;
            while (fine) {
                const Segment *sg = next_segment();
                if (!sg) break;
                const bool live = g == 0 || sg->nq - sg->node0 > a.tile_nodes;
                bool add = false;
                while (true) {
                    const uint32_t vs = steps % H::kNV, buf = steps % kPlaces;
                    if (!(fine = waited(a, sh, &sh.v_ready[vs], (steps / H::kNV) & 1))) break;
                    const volatile Step &info = sh.info[steps % kInfo];
                    const bool page = __shfl_sync(0xffffffffu, info.j, 0) >= 0;
                    if (!(fine = waited(a, sh, &sh.p_full[g][buf], (steps / kPlaces) & 1))) break;
                    tc_fence_after();
                    const uint32_t p = tmem + H::col_s(g, steps);
                    if (issuer) {
                        if (page && live) {
                            const uint32_t vd = tc_desc_mn(v0 + vs * kPageBytes, 8192);
#pragma unroll
                            for (int i = 0; i < 4 * kParts; i++)  // 16 tokens each, part by part
                                tc_mma_ta(d, p + 8 * i, vd + 128 * (i & 3), kIdescO, add || i > 0);
                        }
                        tc_commit(&sh.o_done[g][buf]);
                        tc_commit(&sh.v_free[vs]);
                    }
                    steps++;
                    add = true;
                    if (!page) break;
                }
            }
        }
    } else {
        // ================= values that are not finite =================
        bool fine = true;
        while (fine && next_segment()) {
            bool end = false;
            while (fine && !end) {
                const uint32_t vs = steps % H::kNV;
                if (!(fine = waited(a, sh, &sh.v_full[vs], (steps / H::kNV) & 1))) break;
                const volatile Step &info = sh.info[steps % kInfo];
                const bool edge = info.edge != 0;
                end = info.j < 0;
                if (edge) {
                    uint64_t bad = 0;
                    uint8_t *tile = sh.v[vs];
#pragma unroll 1
                    for (int i0 = 0; i0 < 32; i0 += 8) {  // four rows of a channel half at a time
                        uint4 x[8];
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            x[i] = *reinterpret_cast<const uint4 *>(tile + (i0 + i) * 512 + 16 * lane);
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const uint32_t most = T::max2_nan(
                                T::max2_nan(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                T::max2_nan(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
                            const float2 f = T::unpack(most);
                            const bool wrong = !(f.x < INFINITY && f.y < INFINITY);
                            if (wrong)
                                *reinterpret_cast<uint4 *>(tile + (i0 + i) * 512 + 16 * lane) =
                                    make_uint4(0, 0, 0, 0);
                            const uint32_t who = __ballot_sync(0xffffffffu, wrong);
                            if (who) {
                                for (int q = 0; q < 4; q++)
                                    if ((who >> (8 * q)) & 0xffu) bad |= 1ull << (((i0 + i) & 15) * 4 + q);
                            }
                        }
                    }
                    if (lane == 0) *reinterpret_cast<volatile uint64_t *>(&sh.bad[vs]) = bad;
                    fence_proxy_async();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.v_ready[vs]);
                steps++;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (stopped(sh)) {  // leave nothing in flight (a warp may have been through before another's wait ran out)
        const uint64_t bound = drain_bound_ns(a.wait_ns);
        bool done = true;
        if (warp == H::kCopy && lane == 0) {
            if (segs > 0) done = mbar_drain(&sh.q_full, (segs - 1) & 1, bound);
            for (uint32_t i = 0; i < H::kNK && i < steps + keys; i++) {
                const uint32_t last = steps + keys - 1 - i;
                done &= mbar_drain(&sh.k_full[last % H::kNK], (last / H::kNK) & 1, bound);
            }
            for (uint32_t i = 0; i < H::kNV && i < steps; i++) {
                const uint32_t last = steps - 1 - i;
                done &= mbar_drain(&sh.v_full[last % H::kNV], (last / H::kNV) & 1, bound);
            }
        } else if (issuer) {
            uint64_t *bar = &sh.drain[warp - H::kScores];
            tc_commit(bar);
            done = mbar_drain(bar, 0, bound);
        }
        if (!done) raise_error(a.err, FFD_ERRBIT_TIMEOUT);
        __syncthreads();
    }
    __syncwarp();
    if (warp == 0) tmem_free(tmem, 512);
}

// The cache's rows as a 3-D tensor {64 channels, rows, 2 channel halves}; a copy takes a page's 64 rows
// and lands them as two tiles of 64 x 128 B with the 128-byte swizzle.
bool page_map(CUtensorMap *map, const void *ptr, uint64_t rows, int dtype) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, rows, 2};
    const cuuint64_t strides[2] = {kD * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)kPage, 2};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(map,
              dtype == FFD_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a tensor {channels, heads, rows}; a copy takes half of the channels of G heads and `nodes`
// rows and lands them as rows of 128 B, node by node.
bool query_map(CUtensorMap *map, const AttnArgs &a, int dtype) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {kD, (cuuint64_t)a.Hq, (cuuint64_t)a.total_q};
    const cuuint64_t strides[2] = {kD * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)a.tile_nodes};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(map,
              dtype == FFD_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<uint16_t *>(a.q), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int kTiles, int kParts>
cudaError_t launch(const Params &prm, const Plan &pl, cudaStream_t stream) {
    static int smem_set[kMaxDevicesTracked];
    constexpr int bytes = sizeof(Shared<kTiles>) + 1024;
    cudaError_t e = raise_smem_limit(tree_kernel<T, kTiles, kParts>, bytes, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = pl.ctas;
    cfg.blockDim = Shape<kTiles>::kThreads;
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    // CTAs that share an item wait for each other's records: all of them must be resident
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_kernel<T, kTiles, kParts>, prm);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int tree_slots() { return kSlots; }
size_t tree_record_bytes(int tiles) {
    return (tiles == 1 ? Shape<1>::kRecord : Shape<2>::kRecord) * sizeof(float);
}

cudaError_t launch_tree_attention(const AttnArgs &a, const Plan &pl, int dtype, cudaStream_t stream) {
    Params prm;
    const uint64_t rows = (uint64_t)a.P * a.Hkv * kPage;
    if (!query_map(&prm.tm_q, a, dtype) || !page_map(&prm.tm_k, a.k, rows, dtype) ||
        !page_map(&prm.tm_v, a.v, rows, dtype))
        return cudaErrorInvalidValue;
    prm.a = a;
    char *ws = reinterpret_cast<char *>(a.err);
    prm.records = reinterpret_cast<float *>(ws + pl.records);
    prm.tickets = reinterpret_cast<int *>(ws + pl.tickets);
    auto run = [&](auto type) {
        using T = decltype(type);
        if (pl.tiles == 1) return launch<T, 1, 2>(prm, pl, stream);
        return pl.groups == 1 ? launch<T, 2, 2>(prm, pl, stream) : launch<T, 2, 1>(prm, pl, stream);
    };
    return dtype == FFD_DTYPE_BF16 ? run(Bf16{}) : run(F16{});
}

}  // namespace tree
}  // namespace ffd
