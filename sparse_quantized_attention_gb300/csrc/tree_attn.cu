// tree_attn.cu -- attention of a tree of drafted tokens over the 16-bit cache on the fifth-generation
// tensor cores (ffd_tree_attention in ffd.h).
//
// The query rows of a (sequence, KV head), nq nodes x G heads, are taken kRows = 128 or 256 at a time: an
// item is one such group of rows over the pages that any of them sees. The pages of all items,
// concatenated with what each item costs besides, are cut into equal contiguous ranges, one per CTA (one per
// SM). CTAs that share an item write their parts as records and, once all have come to their range's end, join
// a part of its rows and channels each. In steps of one page (two tiles) or two pages (one tile) a CTA
// computes for each tile of 128 rows
//   S = Q K^T   (M 128, N 64 or 128, K 128; both operands in shared memory, S in tensor memory),
//   P = 2^(S - m) in the inputs' type against a reference m that follows the row's maximum lazily: it is
//       raised, and O rescaled, only when a score passes it by 2^8,
//   O += P V    (M 128, N 128, K 64 a page; P in tensor memory over S, V in shared memory, O in tensor memory).
// Both K and V lie in shared memory as the cache holds them, tokens by channels: K is read along its rows,
// V across them.
//
// Roles: a copy warp lists the pages and fetches them (TMA), running on into the next item while this one
// ends; one warp a tile issues its matrix instructions; four warps a tile do its softmax, a row a thread;
// one warp looks through V where rows see different tokens: a token that some row does not see may hold
// an infinity or a NaN, which a probability of 0 would not silence, so it is zeroed and the rows that do
// see it are marked.
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
constexpr int kInfo = 8;         // steps whose pages are kept
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
    static constexpr int kSoft = 4 * kTiles;               // softmax warps
    static constexpr int kThreads = 32 * (kSoft + 4);      // copy, two issuers, cleaner
    static constexpr int kStep = kTiles == 1 ? 2 : 1;      // pages of a step
    static constexpr int kNK = kTiles == 1 ? 3 : 4;        // steps' K in shared memory
    static constexpr int kNV = 5;                          // pages' V
    static constexpr int kRecord = 130 * kRows;            // floats of a joined item: o[128][row], m, l
    // tensor memory columns of S (P over its first half): a tile has two places in turn
    static __device__ __forceinline__ uint32_t col_s(int g, uint32_t step) {
        return 64 * kStep * (2 * g + (step & 1));
    }
};

struct Step {  // a step's pages: block indexes (first -1: the segment's end, second -1: one page)
    int j0, j1;
    int edge;  // some row does not see all of it
};

struct Cut {  // an item that several CTAs share
    int p0, p1;          // the CTAs, first and last
    int row0, rows;      // its group's first row, rows of it (and of later groups)
    int h, t0;
};

template <int kTiles>
struct Shared {
    using H = Shape<kTiles>;
    uint8_t q[kTiles][2 * 16384];               // tile: channels 0-63, then 64-127
    uint8_t k[H::kNK][H::kStep * kPageBytes];   // the same for a step's tokens
    uint8_t v[H::kNV][kPageBytes];              // the same for 64 tokens
    uint32_t bits[kMaxNodes / 32][H::kRows];    // nodes that a row sees
    int parent[kTiles][kMaxNodes];
    uint64_t k_full[H::kNK], k_free[H::kNK];
    uint64_t v_full[H::kNV], v_ready[H::kNV], v_free[H::kNV];
    uint64_t q_full[kTiles], s_full[kTiles][2], p_full[kTiles][2], o_done[kTiles], drain[kTiles];
    uint64_t bad[H::kNV];                       // tokens of a page whose V is not finite
    Step info[kInfo];
    uint32_t tmem, aborted;
    int scan[H::kThreads / 32];
    int pre[H::kThreads];                       // weight of all items before each chunk of sequences
    Cut cut[2];                                 // the first item, if it began before, and the last, if it goes on
};

struct Params {
    CUtensorMap tm_k, tm_v;
    AttnArgs a;
    float *records;
    int *tickets;
};

// x / G for 0 <= x < 2^29.
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

template <int kRows>
__device__ __forceinline__ int item_groups(const AttnArgs &a, const Seq &s) {
    return (s.nq * a.G + kRows - 1) / kRows;
}

// Positions of an item's rows: at least lo, at most hi. A node's position is not known here; its
// index bounds its depth.
template <int kRows>
__device__ __forceinline__ void item_span(const AttnArgs &a, const Seq &s, int rt, int &lo, int &hi) {
    const int rows = s.nq * a.G;
    const int r1 = (rt + 1) * kRows < rows ? (rt + 1) * kRows : rows;
    lo = s.first() + (a.parents ? 0 : div_g(a, rt * kRows));
    hi = s.first() + div_g(a, r1 - 1);
}

// Pages that the rows of item group rt of a sequence see: the first, and how many.
template <int kRows>
__device__ __forceinline__ void item_pages(const AttnArgs &a, const Seq &s, int rt, int &fp, int &np) {
    int lo, hi;
    item_span<kRows>(a, s, rt, lo, hi);
    fp = a.window > 0 && lo >= a.window ? (lo - a.window + 1) >> 6 : 0;
    np = hi < 0 ? 0 : (hi >> 6) - fp + 1;
}

// What one item weighs: `lead` before its first page and one for each; 0 behind the last one.
template <int kRows>
__device__ __forceinline__ int item_weight(const AttnArgs &a, const Seq &s, int rt) {
    if (rt >= item_groups<kRows>(a, s)) return 0;
    int fp, np;
    item_pages<kRows>(a, s, rt, fp, np);
    return np > 0 ? np + a.lead : 0;
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
template <int kRows>
__device__ __forceinline__ int head_weight(const AttnArgs &a, const Seq &s, int lane) {
    int sum = 0;
    for (int rt = 0; rt < item_groups<kRows>(a, s); rt += 32) sum += item_weight<kRows>(a, s, rt + lane);
    return __reduce_add_sync(0xffffffffu, sum);
}

// A CTA's way through its range of weight [c0, c1): one segment (a run of an item's pages) after another.
template <int kRows>
struct Walk {
    int x, c1;              // where the segment begins in the cut's scale, the range's end
    int b, h, rt, into;     // sequence, KV head, group of rows; weight of the item before x
    Seq s;
    int fp, np, item;       // the item's pages; its first page in the cut's scale
    int at, cnt;            // the segment's pages: at .. at + cnt - 1 of the item's

    // The segment at x; false at the range's end.
    __device__ __forceinline__ bool segment(const AttnArgs &a) {
        if (x >= c1) return false;
        item_pages<kRows>(a, s, rt, fp, np);
        item = x - into + a.lead;
        at = into > a.lead ? into - a.lead : 0;
        cnt = (np < c1 - item ? np : c1 - item) - at;
        return cnt > 0;  // else the item's pages are the next CTA's
    }
    __device__ __forceinline__ void next(const AttnArgs &a) {
        x = item + at + cnt;
        into = 0;
        if (x >= c1) return;
        do {
            if (++rt >= item_groups<kRows>(a, s)) {
                rt = 0;
                if (++h >= a.Hkv) {
                    h = 0;
                    do s = seq_of(a, ++b, false);
                    while (s.nq == 0);
                }
            }
            item_pages<kRows>(a, s, rt, fp, np);
        } while (np == 0);
    }
};

// Bounded waits: once one runs out the CTA stops (aborted) and drains what is in flight.
template <class S>
__device__ __forceinline__ bool stopped(const S &sh) {
    return *reinterpret_cast<const volatile uint32_t *>(&sh.aborted) != 0;
}
template <class S>
__device__ __forceinline__ bool wait_long(const AttnArgs &a, S &sh, uint64_t *bar, uint32_t parity) {
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

template <class T, int kTiles>
__global__ void __launch_bounds__(Shape<kTiles>::kThreads, 1)
    tree_kernel(const __grid_constant__ Params prm) {
    using H = Shape<kTiles>;
    constexpr int kRows = H::kRows, kThreads = H::kThreads, kCtaWarps = kThreads / 32;
    constexpr int kStep = H::kStep;
    constexpr uint32_t kIdescS128 = tc_idesc_f16(128, 128) | Idesc<T>::kType;
    constexpr uint32_t kIdescS64 = tc_idesc_f16(128, 64) | Idesc<T>::kType;
    constexpr uint32_t kIdescO = tc_idesc_f16(128, 128) | Idesc<T>::kType | kTcBMn;
    extern __shared__ uint8_t raw[];
    using Sh = Shared<kTiles>;
    Sh &sh = *reinterpret_cast<Sh *>(align_shared<1024>(raw));
    static_assert(sizeof(Sh) + 1024 <= 232448, "shared memory per CTA");
    const AttnArgs &a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    __syncwarp();
    if (warp == 0) tmem_alloc(&sh.tmem, 512);
    if (tid == 0) {
        sh.aborted = 0;
        sh.cut[0].p0 = sh.cut[1].p0 = -1;
        for (int i = 0; i < H::kNK; i++) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_free[i], kTiles);
        }
        for (int i = 0; i < H::kNV; i++) {
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_ready[i], 1);
            mbar_init(&sh.v_free[i], kTiles);
        }
        for (int g = 0; g < kTiles; g++) {
            mbar_init(&sh.q_full[g], 4);
            for (int j = 0; j < 2; j++) {
                mbar_init(&sh.s_full[g][j], 1);
                mbar_init(&sh.p_full[g][j], 4);
            }
            mbar_init(&sh.o_done[g], 1);
            mbar_init(&sh.drain[g], 1);
        }
        fence_barrier_init();
    }
    // ---- weight of the items before each chunk of sequences: a warp for each of a few, else a thread
    const bool few = a.B <= 4 * kCtaWarps;
    const int chunk = few ? 1 : (a.B + kThreads - 1) / kThreads;
    int own = 0;
    bool empty = false;  // some sequence's rows see nothing
    if (few) {
        for (int b = warp; b < a.B; b += kCtaWarps) {
            const Seq s = seq_of(a, b, blockIdx.x == 0 && lane == 0);
            const int w = head_weight<kRows>(a, s, lane);
            if (lane == 0) sh.pre[b] = w * a.Hkv;
            empty |= s.n == 0 && s.nq > 0;
        }
    } else {
        for (int b = tid * chunk; b < (tid + 1) * chunk && b < a.B; b++) {
            const Seq s = seq_of(a, b, blockIdx.x == 0);
            int w = 0;
            for (int rt = 0; rt < item_groups<kRows>(a, s); rt++) w += item_weight<kRows>(a, s, rt);
            own += w * a.Hkv;
            empty |= s.n == 0 && s.nq > 0;
        }
    }
    empty = __syncthreads_or(empty);
    if (few && tid < a.B) own = sh.pre[tid];
    const int inc = lane_scan(own, lane);
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    const int of_warp = lane_scan(lane < kCtaWarps ? sh.scan[lane] : 0, lane);
    const int total = __shfl_sync(0xffffffffu, of_warp, 31);
    const int warps = __shfl_sync(0xffffffffu, of_warp, warp == 0 ? 0 : warp - 1);
    sh.pre[tid] = (warp == 0 ? 0 : warps) + inc - own;
    if (empty) {
        for (int u = blockIdx.x; u < a.B * a.Hkv; u += gridDim.x) {
            const int b = u / a.Hkv, h = u - b * a.Hkv;
            const Seq s = seq_of(a, b, false);
            if (s.n > 0) continue;
            for (int k = tid; k < s.nq * a.G * 16; k += kThreads) {
                const int r = k >> 4, i = div_g(a, r);
                const int64_t at = (int64_t)(s.t0 + i) * a.Hq + h * a.G + r - i * a.G;
                reinterpret_cast<uint4 *>(a.out + at * kD)[k & 15] = make_uint4(0, 0, 0, 0);
                if (a.lse && (k & 15) == 0) a.lse[at] = -INFINITY;
            }
        }
    }
    const int ncta = total < (int)gridDim.x ? total : (int)gridDim.x, cta = blockIdx.x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (cta >= ncta) {
        __syncwarp();
        if (warp == 0) tmem_free(sh.tmem, 512);
        return;
    }
    const uint32_t tmem = sh.tmem;
    Walk<kRows> w;
    w.x = (int)((int64_t)total * cta / ncta);
    w.c1 = (int)((int64_t)total * (cta + 1) / ncta);
    {   // ---- where the range begins
        int lo = 0, hi = kThreads;  // the last chunk of sequences that begins at or before x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sh.pre[mid] <= w.x) lo = mid;
            else hi = mid;
        }
        int rem = w.x - sh.pre[lo], hp = 1;
        for (w.b = lo * chunk; w.b < a.B; w.b++) {
            w.s = seq_of(a, w.b, false);
            hp = head_weight<kRows>(a, w.s, lane);
            if (rem < hp * a.Hkv) break;
            rem -= hp * a.Hkv;
        }
        w.h = rem / hp;
        rem -= w.h * hp;
        for (w.rt = 0;; w.rt += 32) {  // 32 items at a time
            const int wt = item_weight<kRows>(a, w.s, w.rt + lane), sum = lane_scan(wt, lane);
            const uint32_t past = __ballot_sync(0xffffffffu, sum > rem);
            if (past) {
                const int k = __ffs(past) - 1;
                rem -= __shfl_sync(0xffffffffu, sum - wt, k);
                w.rt += k;
                break;
            }
            rem -= __shfl_sync(0xffffffffu, sum, 31);
        }
        w.into = rem;
    }

    uint32_t steps = 0, vsteps = 0, turns = 0;  // so far: steps and V pages (ends among them), P V products
    if (warp < H::kSoft) {
        // ================= softmax of tile grp, one row a thread =================
        const int grp = warp >> 2, r = tid & (kTile - 1);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t to = tmem + lanes + kColO + grp * 128;
        const float fs = a.factor;
        bool run = true;  // once a wait has run out, only the tickets are still taken
        for (; w.segment(a); w.next(a)) {
            const Seq s = w.s;
            const int h = w.h, first = s.first();
            const int row0 = w.rt * kRows, rows = s.nq * a.G - row0;  // rows: of this item and later
            const bool active = grp == 0 || rows > kTile;
            const bool begins = w.at == 0, complete = begins && w.cnt == w.np;
            const int rr = row0 + grp * kTile + r, qi = div_g(a, rr);
            const bool have = qi < s.nq;
            // ---- queries, half a warp a row (the last item's scores have all been formed)
            if (active && run) {
                const int j = lane & 15;  // channels 8 j .. 8 j + 7
#pragma unroll
                for (int k0 = 0; k0 < 16; k0 += 8) {
                    uint4 got[8];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const int tr = 32 * (warp & 3) + 2 * (k0 + k) + (lane >> 4);
                        const int row = row0 + grp * kTile + tr, i = div_g(a, row);
                        got[k] = make_uint4(0, 0, 0, 0);
                        if (i < s.nq)
                            got[k] = __ldg(reinterpret_cast<const uint4 *>(
                                               a.q + (int64_t)(s.t0 + i) * a.q_stride +
                                               (h * a.G + row - i * a.G) * kD) + j);
                    }
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const int tr = 32 * (warp & 3) + 2 * (k0 + k) + (lane >> 4);
                        *reinterpret_cast<uint4 *>(sh.q[grp] + (j >> 3) * 16384 + tr * 128 +
                                                   (((j & 7) ^ (tr & 7)) << 4)) = got[k];
                    }
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[grp]);
            // ---- the nodes that the row sees, and its position
            int pos = first + qi;
            const bool treed = a.parents && (w.fp + w.at + w.cnt) * kPage > first;
            if (run && a.parents && (treed || a.window > 0)) {
                for (int i = r; i < s.nq; i += kTile) {
                    int p = __ldg(a.parents + s.t0 + i);
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
                const int t0 = 64 * j;
                if (!a.parents) return upto(pos - t0) & ~upto(from - t0);
                uint64_t see = upto(first - 1 - t0) & ~upto(from - t0);
                const int x = t0 - first;  // the page's first token as a node
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
            bool any = false, far = false, tainted = false;
            while (run) {
                const uint32_t buf = steps & 1;
                if (!waited(a, sh, &sh.s_full[grp][buf], (steps >> 1) & 1)) break;
                tc_fence_after();
                const volatile Step &info = sh.info[steps % kInfo];
                const int j0 = info.j0, j1 = info.j1, edge = info.edge;
                const uint32_t ts = tmem + lanes + H::col_s(grp, steps);
                steps++;
                if (j0 < 0) {  // arrived at like any other step, so that the phases go by steps
                    vsteps++;
                    if (lane == 0) mbar_arrive(&sh.p_full[grp][buf]);
                    break;
                }
                const bool both = kStep == 2 && j1 >= 0;
                if (active) {
                    uint64_t see0 = ~0ull, see1 = ~0ull;
                    if (edge) {
                        see0 = visible(j0);
                        if (both) see1 = visible(j1);
                    }
                    // S by pages, 64 columns; of two pages the second is read twice
                    auto page = [&](uint32_t (&x)[64], int n) {
                        __syncwarp();
                        tmem_load32(reinterpret_cast<uint32_t(&)[32]>(x[0]), ts + 64 * n);
                        tmem_load32(reinterpret_cast<uint32_t(&)[32]>(x[32]), ts + 64 * n + 32);
                        tc_wait_load();
                        if (edge) {
                            const uint64_t see = n ? see1 : see0;
                            const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
                            for (int c = 0; c < 32; c++) {
                                if (!((lo >> c) & 1u)) x[c] = 0xff800000u;
                                if (!((hi >> c) & 1u)) x[32 + c] = 0xff800000u;
                            }
                        }
                    };
                    uint32_t x[64];
                    float top = -INFINITY;
                    auto largest = [&]() {
                        float t[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 64; c += 8)
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                t[e] = fmaxf(t[e], fmaxf(__uint_as_float(x[c + 2 * e]),
                                                         __uint_as_float(x[c + 2 * e + 1])));
                        top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                    };
                    if (both) {
                        page(x, 1);
                        largest();
                    }
                    page(x, 0);
                    largest();
                    top *= fs;
                    const bool raise = top > limit;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float mn = raise ? top : m;
                        const float al = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
                        m = mn;
                        limit = m + (is_far(m) ? 0.0f : kLazy);
                        l *= al;
                        far = __any_sync(0xffffffffu, is_far(m));
                        if (any) {
                            // the last step's P V (a stop is met at the next wait)
                            waited(a, sh, &sh.o_done[grp], (turns - 1) & 1);
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
                    auto powers = [&](int n) {
                        if (far) {
#pragma unroll
                            for (int c = 0; c < 64; c++)
                                x[c] = __float_as_uint(__fmul_rn(__uint_as_float(x[c]), fs));
                        }
                        uint32_t p[32];
#pragma unroll
                        for (int c = 0; c < 32; c++) {
                            float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]),
                                                              __uint_as_float(x[2 * c + 1])), f2, s2);
                            e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                            if (c & 1) l3 = __fadd2_rn(l3, e);
                            else l2 = __fadd2_rn(l2, e);
                            p[c] = T::pack(e.x, e.y);
                        }
                        __syncwarp();
                        tmem_store32(ts + 32 * n, p);
                    };
                    powers(0);  // P's first 32 columns lie over S's first half, which has been read
                    if (both) {
                        page(x, 1);
                        powers(1);
                    }
                    l += (l2.x + l2.y) + (l3.x + l3.y);
                    if (edge) {
                        for (int n = 0; n < (both ? 2 : 1); n++) {
                            const uint32_t vs = (vsteps + n) % H::kNV;
                            if (!waited(a, sh, &sh.v_ready[vs], ((vsteps + n) / H::kNV) & 1)) break;
                            tainted |= (*reinterpret_cast<volatile uint64_t *>(&sh.bad[vs]) &
                                        (n ? see1 : see0)) != 0;
                        }
                    }
                    tc_wait_store();
                    any = true;
                }
                vsteps += both ? 2 : 1;
                turns++;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[grp][buf]);
            }
            if (any) {  // the last step's P V
                waited(a, sh, &sh.o_done[grp], (turns - 1) & 1);
                tc_fence_after();
            }
            run = !named_barrier_or(3, kRows, !run || stopped(sh));

            // ---- the segment's results (a whole item's rows by way of the tile's queries, which are
            // read no more, so that lines of out are written whole)
            if (active && run) {
                const float inv = tainted ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
                float *row = prm.records + (int64_t)(kSlots * cta + begins) * H::kRecord + grp * kTile + r;
                uint8_t *stage = sh.q[grp];
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
                    if (complete) {
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                y[k] = T::pack(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                               __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4 *>(stage + r * 256 + (((4 * c + e) ^ (r & 7)) << 4)) =
                                make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else if (have) {
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            row[(32 * c + e) * kRows] = tainted ? NAN : __uint_as_float(o[e]);
                    }
                }
                if (complete) {
                    __syncwarp();
#pragma unroll 4
                    for (int k = 0; k < 16; k++) {
                        const int q = 32 * (warp & 3) + 2 * k + (lane >> 4), c = lane & 15;
                        const int i = div_g(a, row0 + grp * kTile + q);
                        if (i < s.nq)
                            *reinterpret_cast<uint4 *>(
                                a.out + ((int64_t)(s.t0 + i) * a.Hq + h * a.G + row0 + grp * kTile + q -
                                         i * a.G) * kD + 8 * c) =
                                *reinterpret_cast<const uint4 *>(stage + q * 256 + ((c ^ (q & 7)) << 4));
                    }
                    __syncwarp();
                }
                if (have) {
                    if (!complete) row[128 * kRows] = m, row[129 * kRows] = l;
                    else if (a.lse)
                        a.lse[(int64_t)(s.t0 + qi) * a.Hq + h * a.G + rr - qi * a.G] = lse_of(m - kShift, l);
                }
            }
            if (!complete) {  // joined below
                const int p0 = (int)(((int64_t)(w.item + 1) * ncta - 1) / total);
                const int p1 = (int)(((int64_t)(w.item + w.np) * ncta - 1) / total);
                if (tid == 0) sh.cut[begins] = Cut{p0, p1, row0, rows, h, s.t0};
                named_barrier_sync(3, kRows);
                if (tid == 0) add_acq_rel_gpu(prm.tickets + p0, 1);
            }
        }
        // ---- items that several CTAs share: all of them join a part of the rows and channels each
        named_barrier_sync(3, kRows);
#pragma unroll 1
        for (int e = 0; e < 2; e++) {
            const Cut c = sh.cut[e];
            if (c.p0 < 0) continue;
            const int n = c.p1 - c.p0 + 1, place = cta - c.p0;
            if (tid == 0) {
                const uint64_t t0 = globaltimer_ns();
                bool ok = true;
                while (ok && ld_acquire_gpu(prm.tickets + c.p0) < n) ok = globaltimer_ns() - t0 <= a.wait_ns;
                if (!ok) raise_error(a.err, FFD_ERRBIT_TIMEOUT);
            }
            named_barrier_sync(3, kRows);
            const int used = c.rows < kRows ? c.rows : kRows;
            // a unit is 32 rows, one a lane, and 8 channels; `split` warps share one unit's records
            const int units = 16 * ((used + 31) / 32);
            const int mine = units > place ? (units - place + n - 1) / n : 0;  // units place, place + n, ...
            int split = 1;
            while (2 * split * mine <= H::kSoft && 2 * split <= n) split *= 2;
            const int teams = H::kSoft / split, team = warp / split, part = warp % split;
#pragma unroll 1
            for (int u0 = 0; u0 < mine; u0 += teams) {
                const int unit = place + (u0 + team) * n;
                const bool has = u0 + team < mine;
                const int q = 32 * (unit >> 4) + lane, ch = 8 * (unit & 15);
                float M = -INFINITY, ls = 0.0f, o[8] = {};
                // the loads of five records together
                for (int i0 = part; has && i0 < n; i0 += 5 * split) {
                    float v[5][8], mn[5], ln[5];
#pragma unroll
                    for (int i = 0; i < 5; i++) {
                        const bool in = i0 + i * split < n;
                        const int r = in ? i0 + i * split : i0;
                        // a CTA's record: its second one where the item begins, else its first
                        const float *src =
                            prm.records + (int64_t)(kSlots * (c.p0 + r) + (r == 0)) * H::kRecord + q;
#pragma unroll
                        for (int k = 0; k < 8; k++) v[i][k] = __ldcg(src + (ch + k) * kRows);
                        mn[i] = in ? __ldcg(src + 128 * kRows) : -INFINITY;
                        ln[i] = __ldcg(src + 129 * kRows);
                    }
                    float Mn = M;
#pragma unroll
                    for (int i = 0; i < 5; i++) Mn = fmaxf(Mn, mn[i]);
                    const float al = M == -INFINITY ? 0.0f : ex2_approx(M - Mn);
                    M = Mn;
                    ls *= al;
#pragma unroll
                    for (int k = 0; k < 8; k++) o[k] *= al;
#pragma unroll
                    for (int i = 0; i < 5; i++) {
                        if (mn[i] == -INFINITY) continue;  // nothing in it: o and l are 0
                        const float f = ex2_approx(mn[i] - M);
                        ls = fmaf(f, ln[i], ls);
#pragma unroll
                        for (int k = 0; k < 8; k++) o[k] = fmaf(f, v[i][k], o[k]);
                    }
                }
                if (split > 1) {  // the warps' parts, through the space of the queries (one round of units)
                    float *mem = reinterpret_cast<float *>(sh.q[0]) + 32 * 10 * warp + lane;
                    named_barrier_sync(3, kRows);
#pragma unroll
                    for (int k = 0; k < 8; k++) mem[32 * k] = o[k];
                    mem[32 * 8] = M;
                    mem[32 * 9] = ls;
                    named_barrier_sync(3, kRows);
                    if (part > 0) continue;
                    for (int k = 1; k < split; k++) {
                        const float *from = mem + 32 * 10 * k;
                        const float m1 = from[32 * 8];
                        if (m1 == -INFINITY) continue;
                        const float Mn = fmaxf(M, m1);
                        const float f0 = M == -INFINITY ? 0.0f : ex2_approx(M - Mn), f1 = ex2_approx(m1 - Mn);
                        M = Mn;
                        ls = ls * f0 + from[32 * 9] * f1;
#pragma unroll
                        for (int y = 0; y < 8; y++) o[y] = o[y] * f0 + from[32 * y] * f1;
                    }
                }
                if (has && q < used) {
                    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                    const int i = div_g(a, c.row0 + q), head = c.h * a.G + c.row0 + q - i * a.G;
                    const int64_t at = (int64_t)(c.t0 + i) * a.Hq + head;
                    *reinterpret_cast<uint4 *>(a.out + at * kD + ch) =
                        make_uint4(T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv),
                                   T::pack(o[4] * inv, o[5] * inv), T::pack(o[6] * inv, o[7] * inv));
                    if (a.lse && ch == 0) a.lse[at] = lse_of(M - kShift, ls);
                }
            }
            named_barrier_sync(3, kRows);  // all records have been read
            // the last CTA to come leaves both counters at 0 for the next call
            if (tid == 0 && add_acq_rel_gpu(prm.tickets + kMaxCtas + c.p0, 1) == n - 1)
                prm.tickets[c.p0] = prm.tickets[kMaxCtas + c.p0] = 0;
        }
    } else if (warp == H::kSoft) {
        // ================= copies of the pages =================
        if (lane == 0) {
            prefetch_tensormap(&prm.tm_k);
            prefetch_tensormap(&prm.tm_v);
        }
        bool fine = true;
        for (; fine && w.segment(a); w.next(a)) {
            const int32_t *bt = a.block_table + (int64_t)w.b * a.max_blocks;
            const uint8_t *keep =
                a.keep_in ? a.keep_in + ((int64_t)w.b * a.Hkv + w.h) * a.max_blocks : nullptr;
            const int begin = w.fp + w.at, end = begin + w.cnt;
            int lo, hi;
            item_span<kRows>(a, w.s, w.rt, lo, hi);
            const int seen = a.parents ? lo - 1 : lo;  // tokens up to here are seen by all, but for a window
            const int from = a.window > 0 ? hi - a.window : -1;  // and those behind here
            auto look = [&](int j) {
                int p = -1;
                if (j < end && (!keep || __ldg(keep + j))) {
                    p = __ldg(bt + j);
                    if (p < 0 || p >= a.P) {
                        raise_error(a.err, FFD_ERRBIT_BOUNDS);
                        p = -1;
                    }
                }
                return p;
            };
            auto edge = [&](int j) { return 64 * j + 63 > seen || 64 * j <= from; };
            // A step of one or two pages (j0 < 0: the segment's end).
            auto push = [&](int j0, int p0, int j1, int p1) {
                const uint32_t ks = steps % H::kNK;
                if (steps >= H::kNK && !waited(a, sh, &sh.k_free[ks], (steps / H::kNK - 1) & 1)) return false;
                if (lane == 0) {
                    volatile Step &info = sh.info[steps % kInfo];
                    info.j0 = j0;
                    info.j1 = j1;
                    info.edge = j0 >= 0 && (edge(j0) || (j1 >= 0 && edge(j1)));
                    if (j0 >= 0) {
                        mbar_arrive_expect_tx(&sh.k_full[ks], (j1 >= 0 ? 2 : 1) * kPageBytes);
                        if (kStep == 1) {
                            tma_load_3d(sh.k[ks], &prm.tm_k, 0, (p0 * a.Hkv + w.h) * kPage, 0, &sh.k_full[ks]);
                        } else {
#pragma unroll
                            for (int c = 0; c < 2; c++) {  // channel halves
                                tma_load_3d(sh.k[ks] + c * 16384, &prm.tm_k, 0, (p0 * a.Hkv + w.h) * kPage, c,
                                            &sh.k_full[ks]);
                                if (j1 >= 0)
                                    tma_load_3d(sh.k[ks] + c * 16384 + 8192, &prm.tm_k, 0,
                                                (p1 * a.Hkv + w.h) * kPage, c, &sh.k_full[ks]);
                            }
                        }
                    } else {
                        mbar_arrive(&sh.k_full[ks]);
                    }
                }
                steps++;
                for (int n = 0; n < (j1 >= 0 ? 2 : 1); n++) {
                    const uint32_t vs = vsteps % H::kNV;
                    if (vsteps >= H::kNV && !waited(a, sh, &sh.v_free[vs], (vsteps / H::kNV - 1) & 1))
                        return false;
                    if (lane == 0) {
                        if (j0 >= 0) {
                            mbar_arrive_expect_tx(&sh.v_full[vs], kPageBytes);
                            tma_load_3d(sh.v[vs], &prm.tm_v, 0, ((n ? p1 : p0) * a.Hkv + w.h) * kPage, 0,
                                        &sh.v_full[vs]);
                        } else {
                            mbar_arrive(&sh.v_full[vs]);
                        }
                    }
                    vsteps++;
                }
                return true;
            };
            int ahead = look(begin + lane), held = -1, held_page = 0;  // a page that waits for a second one
            for (int jb = begin; jb < end && fine; jb += 32) {
                const int page = ahead;
                ahead = look(jb + 32 + lane);
                for (uint32_t todo = __ballot_sync(0xffffffffu, page >= 0); todo && fine; todo &= todo - 1) {
                    const int k = __ffs(todo) - 1, p = __shfl_sync(0xffffffffu, page, k);
                    if (kStep == 1) {
                        fine = push(jb + k, p, -1, -1);
                    } else if (held < 0) {
                        held = jb + k;
                        held_page = p;
                    } else {
                        fine = push(held, held_page, jb + k, p);
                        held = -1;
                    }
                }
            }
            if (fine && held >= 0) fine = push(held, held_page, -1, -1);
            if (fine) fine = push(-1, -1, -1, -1);
        }
        if (stopped(sh) && lane == 0) {  // leave nothing in flight
            bool done = true;
            for (uint32_t i = 0; i < H::kNK && i < steps; i++) {
                const uint32_t last = steps - 1 - i;
                done &= mbar_drain(&sh.k_full[last % H::kNK], (last / H::kNK) & 1, drain_bound_ns(a.wait_ns));
            }
            for (uint32_t i = 0; i < H::kNV && i < vsteps; i++) {
                const uint32_t last = vsteps - 1 - i;
                done &= mbar_drain(&sh.v_full[last % H::kNV], (last / H::kNV) & 1, drain_bound_ns(a.wait_ns));
            }
            if (!done) raise_error(a.err, FFD_ERRBIT_TIMEOUT);
        }
    } else if (warp < H::kSoft + 1 + kTiles) {
        // ================= matrix instructions of one tile =================
        // The whole warp goes through the steps, so that operand addresses stay warp-uniform; one lane
        // issues.
        const int g = warp - H::kSoft - 1;
        const bool issuer = elect_one();
        const uint32_t k0 = smem_u32(sh.k[0]), v0 = smem_u32(sh.v[0]);
        const uint32_t qd = tc_desc(smem_u32(sh.q[g]));
        uint32_t items = 0;
        bool fine = true;
        for (; fine && w.segment(a); w.next(a)) {
            const bool live = g == 0 || w.s.nq * a.G - w.rt * kRows > kTile;
            fine = waited(a, sh, &sh.q_full[g], items++ & 1);
            // The scores of the next step. 0 at the segment's end, which the softmax group learns of in the
            // same way; else its pages. Negative: stopped.
            auto next_scores = [&]() {
                const uint32_t ks = steps % H::kNK, d = tmem + H::col_s(g, steps);
                if (!waited(a, sh, &sh.k_full[ks], (steps / H::kNK) & 1)) return -1;
                tc_fence_after();
                const volatile Step &info = sh.info[steps % kInfo];
                int pages = info.j0 < 0 ? 0 : info.j1 < 0 ? 1 : 2;
                pages = __shfl_sync(0xffffffffu, pages, 0);
                const uint32_t kd = tc_desc(k0 + ks * (kStep * kPageBytes));
                if (issuer) {
                    if (pages && live) {
                        const uint32_t idesc = kStep == 2 && pages == 2 ? kIdescS128 : kIdescS64;
#pragma unroll
                        for (int i = 0; i < 8; i++)  // 16 channels each
                            tc_mma(d, qd + (i >> 2) * 1024 + (i & 3) * 2,
                                   kd + (i >> 2) * (512 * kStep) + (i & 3) * 2, idesc, i > 0);
                    }
                    tc_commit(&sh.s_full[g][steps & 1]);
                    tc_commit(&sh.k_free[ks]);
                }
                steps++;
                return pages;
            };
            uint32_t pstep = steps;  // the step whose values come next
            int cur = fine ? next_scores() : -1, nxt = 0;
            if (cur > 0) nxt = next_scores();  // two steps' scores are under way before the first P V
            bool add = false;
            while (cur > 0) {
                fine = false;
                const uint32_t vs0 = vsteps % H::kNV, vs1 = (vsteps + 1) % H::kNV;
                if (!waited(a, sh, &sh.v_ready[vs0], (vsteps / H::kNV) & 1)) break;
                if (cur == 2 && !waited(a, sh, &sh.v_ready[vs1], ((vsteps + 1) / H::kNV) & 1)) break;
                if (!waited(a, sh, &sh.p_full[g][pstep & 1], (pstep >> 1) & 1)) break;
                tc_fence_after();
                const uint32_t p = tmem + H::col_s(g, pstep), d = tmem + kColO + g * 128;
                if (issuer) {
                    if (live) {
                        const uint32_t vd0 = tc_desc_mn(v0 + vs0 * kPageBytes, 8192);
                        const uint32_t vd1 = tc_desc_mn(v0 + vs1 * kPageBytes, 8192);
#pragma unroll
                        for (int i = 0; i < 4; i++)  // 16 tokens each
                            tc_mma_ta(d, p + 8 * i, vd0 + 128 * i, kIdescO, add || i > 0);
                        if (cur == 2) {
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                tc_mma_ta(d, p + 32 + 8 * i, vd1 + 128 * i, kIdescO, true);
                        }
                    }
                    tc_commit(&sh.o_done[g]);
                }
                if (!waited(a, sh, &sh.o_done[g], turns & 1)) break;
                if (issuer) {
                    mbar_arrive(&sh.v_free[vs0]);
                    if (cur == 2) mbar_arrive(&sh.v_free[vs1]);
                }
                vsteps += cur;
                turns++;
                pstep++;
                add = true;
                fine = true;
                const int third = nxt > 0 ? next_scores() : nxt;
                cur = nxt;
                nxt = third;
            }
            if (cur < 0) fine = false;
            if (fine) {  // the end's V place
                fine = waited(a, sh, &sh.v_ready[vsteps % H::kNV], (vsteps / H::kNV) & 1);
                if (fine && issuer) mbar_arrive(&sh.v_free[vsteps % H::kNV]);
                vsteps++;
            }
        }
        if (stopped(sh) && issuer) {
            tc_commit(&sh.drain[g]);
            if (!mbar_drain(&sh.drain[g], 0, drain_bound_ns(a.wait_ns))) raise_error(a.err, FFD_ERRBIT_TIMEOUT);
        }
    } else if (warp == kCtaWarps - 1) {
        // ================= values that are not finite =================
        bool fine = true;
        for (; fine && w.segment(a); w.next(a)) {
            while (true) {
                fine = waited(a, sh, &sh.v_full[vsteps % H::kNV], (vsteps / H::kNV) & 1);
                if (!fine) break;
                const volatile Step &info = sh.info[steps % kInfo];
                const bool end = info.j0 < 0, edge = info.edge != 0;
                const int pages = info.j1 >= 0 ? 2 : 1;
                steps++;
                for (int n = 0; n < pages; n++) {
                    const uint32_t vs = vsteps % H::kNV;
                    if (n > 0 && !(fine = waited(a, sh, &sh.v_full[vs], (vsteps / H::kNV) & 1))) break;
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
                                uint32_t most = T::max2_nan(
                                    T::max2_nan(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                    T::max2_nan(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
                                const float2 f = T::unpack(most);
                                const bool wrong = !(f.x < INFINITY && f.y < INFINITY);
                                if (wrong)
                                    *reinterpret_cast<uint4 *>(tile + (i0 + i) * 512 + 16 * lane) =
                                        make_uint4(0, 0, 0, 0);
                                uint32_t who = __ballot_sync(0xffffffffu, wrong);
                                if (who) {
                                    for (int q = 0; q < 4; q++)
                                        if ((who >> (8 * q)) & 0xffu)
                                            bad |= 1ull << (((i0 + i) & 15) * 4 + q);
                                }
                            }
                        }
                        if (lane == 0) *reinterpret_cast<volatile uint64_t *>(&sh.bad[vs]) = bad;
                        fence_proxy_async();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.v_ready[vs]);
                    vsteps++;
                }
                if (end || !fine) break;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if (warp == 0) tmem_free(tmem, 512);
}

// The cache's rows as a 3-D tensor {64 channels, rows, 2 channel halves}; a copy takes a page's 64 rows of
// `halves` halves and lands them as tiles of 64 x 128 B with the 128-byte swizzle.
bool page_map(CUtensorMap *map, const void *ptr, uint64_t rows, int dtype, uint32_t halves) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, rows, 2};
    const cuuint64_t strides[2] = {kD * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)kPage, halves};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(map,
              dtype == FFD_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int kTiles>
cudaError_t launch(const Params &prm, const Plan &pl, cudaStream_t stream) {
    static int smem_set[kMaxDevicesTracked];
    constexpr int bytes = sizeof(Shared<kTiles>) + 1024;
    cudaError_t e = raise_smem_limit(tree_kernel<T, kTiles>, bytes, smem_set);
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
    e = cudaLaunchKernelEx(&cfg, tree_kernel<T, kTiles>, prm);
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
    if (!page_map(&prm.tm_k, a.k, rows, dtype, pl.tiles == 1 ? 1 : 2) || !page_map(&prm.tm_v, a.v, rows, dtype, 2))
        return cudaErrorInvalidValue;
    prm.a = a;
    char *ws = reinterpret_cast<char *>(a.err);
    prm.records = reinterpret_cast<float *>(ws + pl.records);
    prm.tickets = reinterpret_cast<int *>(ws + pl.tickets);
    if (dtype == FFD_DTYPE_BF16)
        return pl.tiles == 1 ? launch<Bf16, 1>(prm, pl, stream) : launch<Bf16, 2>(prm, pl, stream);
    return pl.tiles == 1 ? launch<F16, 1>(prm, pl, stream) : launch<F16, 2>(prm, pl, stream);
}

}  // namespace tree
}  // namespace ffd
