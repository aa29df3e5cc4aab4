// kv4_chunk.cu -- attention over the 4-bit cache for many query rows (drafted tokens, chunks of a
// prompt) on the fifth-generation tensor cores. Definition in ffd.h.
//
// The query rows of a (sequence, KV head), nq tokens x G heads, are taken 256 at a time: an item is
// one such group of rows over the pages that any of them sees. The pages of all items, concatenated with
// what each item costs besides, are cut into equal contiguous ranges, one per CTA (one per SM), so the
// last CTA ends with the first whatever the causal edges leave; an item cut by a range's end is joined
// by the last of its CTAs.
// Where items are short, whole ones are dealt out instead (a join costs more than the imbalance), if the
// sequences' lengths are even enough.
// For each page of 64 tokens a CTA computes, for its two tiles of 128 rows,
//   S = Q K^T   (M 128, N 64, K 128; f16, both operands in shared memory, S in tensor memory),
//   P = 2^(S - m) in f16 against a reference m that follows the row's maximum lazily: it is raised,
//       and O rescaled, only when a score passes it by 2^8,
//   O += P V    (M 128, N 128, K 64; P in tensor memory, V^T in shared memory, O in tensor memory).
// Roles: a copy warp fetches the pages' records; four warps form K and four V^T tiles of f16 values from
// them; one thread a tile issues its matrix instructions; two groups of four warps, one row a thread,
// do the softmax of one tile each.
//
// What bounds it. A page takes 2040 cycles for two tiles (2048 query tokens over 32768, 32/8 heads:
// 932 us, 1.14 PFLOP/s, 59 % of the measured matrix rate; 1280 cycles are the matrix instructions' own: 8 x
// 48 a tile for S, whose Q is read again from shared memory every time, and 4 x 64 for P V) and 1780
// for one. Within a step the softmax of a row (2020 cycles with both groups at work, 1680 with one) and
// the way S -> P -> P V -> next S through barriers cover each other, but little is left between. Q
// partly in tensor memory (S at 40 cycles an instruction) leaves room for three places of S and
// ties the tiles to each other: 1287 us, when this form took 955. A CTA of 480 threads that reads S once into
// 128 registers forms K and V^T with four warps, and waits for them: 961 us then.
//
// K's rows, and with them the columns of S, P and V^T, are tokens in the order 8 (p % 8) + p / 8:
// then the eight tokens that make 16 bytes of a V^T row come from eight different lanes' loads, and
// neither side of the transposition meets a bank conflict.
#include "kv4_walk.cuh"

namespace ffd {
namespace kv4 {
namespace {

constexpr int kTile = 128;             // rows of a tile
constexpr int kRows = 2 * kTile;       // rows of an item
// 2 x 4 softmax warps, 4 warps forming K, 4 forming V, 2 issuers, copy: 96 registers a thread, 48 bytes spilled
constexpr int kThreads = 608;
constexpr int kCtaWarps = kThreads / 32;
constexpr int kNK = 3, kNV = 3;        // f16 tiles of K and of V^T
constexpr int kNS = 5;                 // record pairs in flight
constexpr int kInfo = 16;              // steps whose page index is kept
constexpr int kRecord = 130 * kRows;   // floats of a joined item: o[128][row], m[row], l[row]
// Records of a CTA: of the item that goes on from before, of the one that begins there; of a group of
// CTAs whose first one this is, where the item begins or goes on.
constexpr int kSlots = 4;
constexpr int kOnce = 8;               // records (133 KB each) that one CTA joins at once
// Tensor memory columns: S of tile g and step j at 64 (2 g + j % 2), its first 32 columns P's place
// once S is read; O of tile g at kColO + 128 g.
constexpr uint32_t kColO = 256;
__device__ __forceinline__ uint32_t col_s(int g, uint32_t step) { return 64 * (2 * g + (step & 1)); }
constexpr uint32_t kIdescS = tc_idesc_f16(128, 64), kIdescO = tc_idesc_f16(128, 128);

struct Shared {
    uint8_t q[2][2 * 16384];           // tile: channels 0-63, then 64-127
    uint8_t k[kNK][2 * 8192];          // the same for 64 rows
    uint8_t v[kNV][16384];             // V^T: 128 channels x 64 tokens
    uint8_t rec[kNS][2 * kRec];        // K record, V record
    uint64_t rec_full[kNS], rec_free[kNS];
    uint64_t k_full[kNK], k_free[kNK], v_full[kNV], v_free[kNV];
    uint64_t s_full[2][2], p_full[2][2];  // [tile][step % 2]: scores stand, probabilities stand
    uint64_t o_done[2], drain[2];         // P V of a tile's step is done
    uint32_t tmem, aborted;
    int info[kInfo];                   // page index of a step, -1: the segment's end
    int scan[2][kCtaWarps], heaviest[kCtaWarps];
    int flag;
    float factor[kRows];               // of the rows' scores
    // weight and number of all items before each chunk of sequences
    int pre[kThreads], pre_items[kThreads];
};
static_assert(sizeof(Shared) + 1024 <= 232448, "shared memory per CTA");

// x / G for 0 <= x < 2^29.
__device__ __forceinline__ int div_g(const AttnArgs &a, int x) {
    return a.G == 1 ? x : (int)__umulhi((uint32_t)x, a.over_g);
}

__device__ __forceinline__ int item_groups(const AttnArgs &a, const Seq &s) {
    return (s.nq * a.G + kRows - 1) / kRows;
}

// Pages that the rows of item group rt of a sequence see: the first, and how many.
__device__ __forceinline__ void item_pages(const AttnArgs &a, const Seq &s, int rt, int &fp,
                                           int &np) {
    const int rows = s.nq * a.G;
    const int r1 = (rt + 1) * kRows < rows ? (rt + 1) * kRows : rows;
    const int lo = s.n - s.nq + div_g(a, rt * kRows), hi = s.n - s.nq + div_g(a, r1 - 1);
    const int first = a.window > 0 && lo >= a.window ? lo - a.window + 1 : 0;
    fp = first >> 6;
    np = hi < 0 ? 0 : (hi >> 6) - fp + 1;
}

// What one item weighs: `lead` before its first page and one for each; 0 behind the last one.
__device__ __forceinline__ int item_weight(const AttnArgs &a, const Seq &s, int rt) {
    if (rt >= item_groups(a, s)) return 0;
    int fp, np;
    item_pages(a, s, rt, fp, np);
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
__device__ __forceinline__ int head_weight(const AttnArgs &a, const Seq &s, int lane) {
    int sum = 0;
    for (int rt = 0; rt < item_groups(a, s); rt += 32) sum += item_weight(a, s, rt + lane);
    return __reduce_add_sync(0xffffffffu, sum);
}

// Whether whole items may be dealt out where the host has found that the block table's width and the
// numbers of rows allow it (it cannot see the lengths): `heaviest` is the greatest of the sequences' mean
// items. The longest-working CTA has at most `rounds` such items; when that is more than an equal share by
// what cutting costs, the lengths are too unequal. Measured, us whole and cut, 8 heads, 4 query heads each:
//   19 sequences of 1024 tokens, their last 9                        31   32
//   18 of them, and one of 32768                                    471   74
//   18 of them, and one of 131072                                  1831  152
//   37 of 512 tokens, their last 64, and one of 16384               560   90
__device__ __forceinline__ bool even_enough(int items, int weight, int heaviest, int ctas) {
    const int rounds = (items + ctas - 1) / ctas, share = items < ctas ? items : ctas;
    const int beyond = rounds * heaviest - (rounds > 1 ? kJoinPagesSeveral : kJoinPages);
    return (int64_t)beyond * share <= weight;
}

// Bounded waits: once one runs out the CTA stops (aborted) and drains what is in flight.
__device__ __forceinline__ bool stopped(const Shared &sh) {
    return *reinterpret_cast<const volatile uint32_t *>(&sh.aborted) != 0;
}
__device__ __forceinline__ bool wait_long(const AttnArgs &a, Shared &sh, uint64_t *bar, uint32_t parity) {
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
__device__ __forceinline__ bool waited(const AttnArgs &a, Shared &sh, uint64_t *bar, uint32_t parity) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_long(a, sh, bar, parity);
    return __all_sync(0xffffffffu, ok);
}

// ---- forming the tiles --------------------------------------------------------------------------
// K: thread t takes word t % 16 of tokens t / 16, t / 16 + 8, ...; row p = 8 (token % 8) + token / 8.
__device__ __forceinline__ void form_k(const uint8_t *rec, uint8_t *tile, int t) {
    const int J = t & 15, r0 = t >> 4;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = r0 + 8 * i;
        const uint32_t w =
            *reinterpret_cast<const uint32_t *>(rec + code_offset(r, J >> 2) + 4 * (J & 3));
        const __half2 p = *reinterpret_cast<const __half2 *>(rec + param_offset(r, J >> 2));
        __half2 v[4];
        decode_word(w, p, v);
        const int row = 8 * r0 + i;  // r = 8 i + r0
        *reinterpret_cast<uint4 *>(tile + (J >> 3) * 8192 + row * 128 + (((J & 7) ^ (row & 7)) << 4)) =
            *reinterpret_cast<const uint4 *>(v);
    }
}

// V^T: thread t takes word J = 4 (t / 32) + t % 32 / 8 of the tokens i * 8 + tg (i < 8), tg = t % 8,
// which are positions 8 tg .. 8 tg + 7: 16 bytes of each of the word's eight channel rows. Tokens
// before `from` and from `valid` on, which no query sees, may hold anything and count as 0.
__device__ __forceinline__ void form_v(const uint8_t *rec, uint8_t *tile, int t, int from, int valid) {
    const int tg = t & 7, J = 4 * (t >> 5) + ((t >> 3) & 3);
    uint32_t out[8][4];  // [channel of the word][token pair]
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = 16 * i + tg;  // tokens r and r + 8: positions 8 tg + 2 i, + 1
        const uint32_t w0 =
            *reinterpret_cast<const uint32_t *>(rec + code_offset(r, J >> 2) + 4 * (J & 3));
        const uint32_t w1 =
            *reinterpret_cast<const uint32_t *>(rec + code_offset(r + 8, J >> 2) + 4 * (J & 3));
        uint32_t p0 = *reinterpret_cast<const uint32_t *>(rec + param_offset(r, J >> 2));
        uint32_t p1 = *reinterpret_cast<const uint32_t *>(rec + param_offset(r + 8, J >> 2));
        if (from > 0 || valid < kPage) {
            p0 = r >= from && r < valid ? p0 : 0u;
            p1 = r + 8 >= from && r + 8 < valid ? p1 : 0u;
        }
        const uint32_t sw = __byte_perm(p0, p1, 0x5410), ow = __byte_perm(p0, p1, 0x7632);
        const __half2 s = *reinterpret_cast<const __half2 *>(&sw);
        const __half2 o = *reinterpret_cast<const __half2 *>(&ow);
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const uint32_t w = __byte_perm(w0, w1, e ? 0x7632 : 0x5410);
            const __half2 v[4] = {__hfma2(code_pair<0>(w), s, o), __hfma2(code_pair<1>(w), s, o),
                                  __hfma2(code_pair<2>(w), s, o), __hfma2(code_pair<3>(w), s, o)};
#pragma unroll
            for (int c = 0; c < 4; c++)
                out[2 * c + e][i] = *reinterpret_cast<const uint32_t *>(&v[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < 8; c++)
        *reinterpret_cast<uint4 *>(tile + (8 * J + c) * 128 + ((tg ^ c) << 4)) =
            make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]);
}

// The item's rows of q into the tiles as scaled f16, half a warp a row, and their scores' factors.
template <class T>
__device__ __forceinline__ void load_queries(const AttnArgs &a, Shared &sh, const Seq &s, int h,
                                             int row0, int rows, int warp, int lane) {
    const int j = lane & 15;  // channels 8 j .. 8 j + 7
    constexpr int kEach = (kRows / 2 + kCtaWarps - 1) / kCtaWarps;
    uint4 got[kEach];  // all loads are under way before the first is waited for
#pragma unroll
    for (int k = 0; k < kEach; k++) {
        const int r = 2 * (warp + k * kCtaWarps) + (lane >> 4), i = div_g(a, row0 + r);
        got[k] = make_uint4(0, 0, 0, 0);
        if (r < rows && i < s.nq)
            got[k] = __ldg(reinterpret_cast<const uint4 *>(
                               static_cast<const uint16_t *>(a.q) + (int64_t)(s.t0 + i) * a.q_stride +
                               (h * a.G + row0 + r - i * a.G) * kD) + j);
    }
#pragma unroll
    for (int k = 0; k < kEach; k++) {
        const int r = 2 * (warp + k * kCtaWarps) + (lane >> 4);
        if (r >= rows) break;  // warp-uniform: rows is even
        const uint4 u = got[k];
        const float2 x0 = T::unpack(u.x), x1 = T::unpack(u.y), x2 = T::unpack(u.z),
                     x3 = T::unpack(u.w);
        float top = fmaxf(fmaxf(fmaxf(fabsf(x0.x), fabsf(x0.y)), fmaxf(fabsf(x1.x), fabsf(x1.y))),
                          fmaxf(fmaxf(fabsf(x2.x), fabsf(x2.y)), fmaxf(fabsf(x3.x), fabsf(x3.y))));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float mul, f;
        query_scale(a, top, mul, f);
        const int tr = r & (kTile - 1);
        *reinterpret_cast<uint4 *>(sh.q[r / kTile] + (j >> 3) * 16384 + tr * 128 +
                                   (((j & 7) ^ (tr & 7)) << 4)) =
            make_uint4(F16::pack(x0.x * mul, x0.y * mul), F16::pack(x1.x * mul, x1.y * mul),
                       F16::pack(x2.x * mul, x2.y * mul), F16::pack(x3.x * mul, x3.y * mul));
        if (j == 0) sh.factor[r] = f;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_kernel(const AttnArgs a, float *records,
                                                                int *tickets) {
    extern __shared__ uint8_t raw[];
    Shared &sh = *reinterpret_cast<Shared *>(align_shared<1024>(raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    __syncwarp();
    if (warp == 0) tmem_alloc(&sh.tmem, 512);
    if (tid == 0) {
        sh.aborted = 0;
        for (int i = 0; i < kNS; i++) {
            mbar_init(&sh.rec_full[i], 1);
            mbar_init(&sh.rec_free[i], 8);
        }
        for (int i = 0; i < kNK; i++) {
            mbar_init(&sh.k_full[i], 4);
            mbar_init(&sh.k_free[i], 2);
        }
        for (int i = 0; i < kNV; i++) {
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.v_free[i], 2);
        }
        for (int i = 0; i < 2; i++) {
            for (int j = 0; j < 2; j++) {
                mbar_init(&sh.s_full[i][j], 1);
                mbar_init(&sh.p_full[i][j], 4);
            }
            mbar_init(&sh.o_done[i], 1);
            mbar_init(&sh.drain[i], 1);
        }
        fence_barrier_init();
    }
    // ---- weight of the items before each chunk of sequences: a warp for each of a few, else a thread
    const bool few = a.B <= 4 * kCtaWarps;
    const int chunk = few ? 1 : (a.B + kThreads - 1) / kThreads;
    int own = 0, own_items = 0, heaviest = 0;
    bool empty = false;  // some rows see nothing: perhaps whole items
    if (few) {
        for (int b = warp; b < a.B; b += kCtaWarps) {
            const Seq s = seq_of(a, b, blockIdx.x == 0);
            const int w = head_weight(a, s, lane), n = item_groups(a, s);
            if (lane == 0) sh.pre[b] = w * a.Hkv, sh.pre_items[b] = n * a.Hkv;
            if (n > 0) heaviest = max(heaviest, (w + n - 1) / n);
            empty |= s.n < s.nq;
        }
    } else {
        for (int b = tid * chunk; b < (tid + 1) * chunk && b < a.B; b++) {
            const Seq s = seq_of(a, b, blockIdx.x == 0);
            const int n = item_groups(a, s);
            int w = 0;
            for (int rt = 0; rt < n; rt++) w += item_weight(a, s, rt);
            own += w * a.Hkv;
            own_items += n * a.Hkv;
            if (n > 0) heaviest = max(heaviest, (w + n - 1) / n);
            empty |= s.n < s.nq;
        }
    }
    if (a.whole_items) {
        heaviest = __reduce_max_sync(0xffffffffu, heaviest);
        if (lane == 0) sh.heaviest[warp] = heaviest;
    }
    empty = __syncthreads_or(empty);
    if (few && tid < a.B) own = sh.pre[tid], own_items = sh.pre_items[tid];
    const int inc = lane_scan(own, lane);
    if (lane == 31) sh.scan[0][warp] = inc;
    int inc_items = 0;
    if (a.whole_items) {
        inc_items = lane_scan(own_items, lane);
        if (lane == 31) sh.scan[1][warp] = inc_items;
    }
    __syncthreads();
    int total, total_items = 0;
    auto prefix = [&](int which, int before, int *pre, int &all) {
        const int of_warp = lane_scan(lane < kCtaWarps ? sh.scan[which][lane] : 0, lane);
        all = __shfl_sync(0xffffffffu, of_warp, 31);
        const int warps = __shfl_sync(0xffffffffu, of_warp, warp == 0 ? 0 : warp - 1);
        pre[tid] = (warp == 0 ? 0 : warps) + before;
    };
    prefix(0, inc - own, sh.pre, total);
    bool whole = false;
    if (a.whole_items) {
        prefix(1, inc_items - own_items, sh.pre_items, total_items);
        heaviest = __reduce_max_sync(0xffffffffu, lane < kCtaWarps ? sh.heaviest[lane] : 0);
        whole = even_enough(total_items, total, heaviest, gridDim.x);
    }
    const bool any_empty = empty;
    if (any_empty) {  // items that see nothing at all
        for (int u = blockIdx.x; u < a.B * a.Hkv; u += gridDim.x) {
            const int b = u / a.Hkv, h = u - b * a.Hkv;
            const Seq s = seq_of(a, b, false);
            for (int rt = 0; rt < item_groups(a, s); rt++) {
                int fp, np;
                item_pages(a, s, rt, fp, np);
                if (np > 0) break;  // later items see more
                for (int k = tid; k < kRows * 64; k += kThreads) {
                    const int r = rt * kRows + (k >> 6), i = div_g(a, r), hq = h * a.G + r - i * a.G;
                    if (i >= s.nq) break;
                    write_pair<T>(a, s.t0 + i, hq, 2 * (k & 63), 0.0f, 0.0f);
                    if (a.lse && (k & 63) == 0) a.lse[(int64_t)(s.t0 + i) * a.Hq + hq] = -INFINITY;
                }
            }
        }
    }
    const int shares = whole ? total_items : total;
    const int ncta = shares < (int)gridDim.x ? shares : (int)gridDim.x;
    const int cta = blockIdx.x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (cta >= ncta) {
        __syncwarp();
        if (warp == 0) tmem_free(sh.tmem, 512);
        return;
    }
    const uint32_t tmem = sh.tmem;
    int c0 = (int)((int64_t)shares * cta / ncta), c1 = (int)((int64_t)shares * (cta + 1) / ncta);
    auto chunk_of = [&](const int *pre, int x) {  // the last chunk of sequences that begins at or before x
        int lo = 0, hi = kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    // ---- where the range begins: sequence b, head h, group rt, `into` the item's weight ----------
    int b = 0, h = 0, rt = 0, into = 0;
    Seq s = {0, 0, 0, 0, 0};
    auto next_item = [&]() {
        if (++rt < item_groups(a, s)) return;
        rt = 0;
        if (++h < a.Hkv) return;
        h = 0;
        do {
            s = seq_of(a, ++b, false);
        } while (s.nq == 0);
    };
    if (whole) {  // items c0 .. c1 - 1: then a range of weight from the first that has some
        const int lo = chunk_of(sh.pre_items, c0), items = c1 - c0;
        int rem = c0 - sh.pre_items[lo], n = 0;
        for (b = lo * chunk; b < a.B; b++) {
            s = seq_of(a, b, false);
            n = item_groups(a, s);
            if (rem < n * a.Hkv) break;
            rem -= n * a.Hkv;
        }
        h = rem / n;
        rt = rem - h * n;
        c0 = c1 = 0;
        int b0 = b, h0 = h, rt0 = rt;
        Seq s0 = s;
        for (int i = 0; i < items; i++) {
            if (i > 0) next_item();
            const int w = item_weight(a, s, rt);
            if (c1 == 0) b0 = b, h0 = h, rt0 = rt, s0 = s;
            c1 += w;
        }
        b = b0, h = h0, rt = rt0, s = s0;
    } else {
        const int lo = chunk_of(sh.pre, c0);
        int rem = c0 - sh.pre[lo], hp = 0;
        for (b = lo * chunk; b < a.B; b++) {
            s = seq_of(a, b, false);
            hp = head_weight(a, s, lane);
            if (rem < hp * a.Hkv) break;
            rem -= hp * a.Hkv;
        }
        h = rem / hp;
        rem -= h * hp;
        for (;; rt += 32) {  // 32 items at a time
            const int w = item_weight(a, s, rt + lane), upto = lane_scan(w, lane);
            const uint32_t past = __ballot_sync(0xffffffffu, upto > rem);
            if (past) {
                const int k = __ffs(past) - 1;
                rem -= __shfl_sync(0xffffffffu, upto - w, k);
                rt += k;
                break;
            }
            rem -= __shfl_sync(0xffffffffu, upto, 31);
        }
        into = rem;
    }

    // so far in the whole kernel, per role: steps (segments' ends among them), and pages (V tiles and
    // P V products)
    uint32_t steps = 0, vsteps = 0, turns = 0;
    for (int x = c0; x < c1;) {
        int fp, np;
        item_pages(a, s, rt, fp, np);
        const int first = x - into + a.lead;  // the item's first page in the cut's scale
        const int at = into > a.lead ? into - a.lead : 0;
        const int cnt = (np < c1 - first ? np : c1 - first) - at;
        if (cnt <= 0) break;  // the item's pages are the next CTA's
        const int j0 = fp + at, j1 = j0 + cnt;
        const int row0 = rt * kRows, rows = s.nq * a.G - row0;  // rows: of this item and later
        const bool two = rows > kTile;
        const bool begins = at == 0, complete = begins && cnt == np;

        // ---- queries
        const int grp = warp >> 2;  // 0, 1: softmax group
        const int r = tid & (kTile - 1);
        const int rr = row0 + grp * kTile + r, qi = div_g(a, rr);
        const bool have = grp < 2 && qi < s.nq;
        if (!stopped(sh)) {
            load_queries<T>(a, sh, s, h, row0, two ? kRows : kTile, warp, lane);
            fence_proxy_async();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        bool run = !stopped(sh);
        __syncthreads();  // nobody stops between the reading of it and this
        const float fs = grp < 2 ? sh.factor[grp * kTile + r] : 0.0f;

        float m = -INFINITY, limit = -INFINITY, l = 0.0f;  // limit: a larger score raises m
        bool any = false, far = false;
        if (run && grp < 2) {
            // ================= softmax of tile grp, one row a thread =================
            const bool active = grp == 0 || two;
            const uint32_t lanes = (uint32_t)(warp & 3) << 21;
            const uint32_t to = tmem + lanes + kColO + grp * 128;
            const int pos = s.n - s.nq + qi;
            const int from = a.window > 0 ? pos - a.window : -1;
            // positions of the tile's first and last row
            const int lo = s.n - s.nq + div_g(a, row0 + grp * kTile);
            const int hi = s.n - 1 < lo + (kTile - 1) / a.G + 1 ? s.n - 1 : lo + (kTile - 1) / a.G + 1;
            while (true) {
                const uint32_t buf = steps & 1;
                if (!waited(a, sh, &sh.s_full[grp][buf], (steps >> 1) & 1)) break;
                tc_fence_after();
                const int j = *reinterpret_cast<volatile int *>(&sh.info[steps % kInfo]);
                const uint32_t ts = tmem + lanes + col_s(grp, steps);
                steps++;
                if (j < 0) {  // arrived at like any other step, so that the phases go by steps
                    if (lane == 0) mbar_arrive(&sh.p_full[grp][buf]);
                    break;
                }
                if (active) {
                    // S in halves of 32 columns, the first read twice: a row's 64 scores at once would
                    // leave no registers for the warps that form the tiles
                    const int t0 = 64 * j;
                    const bool open = t0 + 63 <= lo && (a.window == 0 || t0 > hi - a.window);
                    auto half = [&](uint32_t (&x)[32], int n) {
                        __syncwarp();
                        tmem_load32(x, ts + 32 * n);
                        tc_wait_load();
                        if (!open) {
#pragma unroll
                            for (int c = 0; c < 32; c++) {
                                const int k = t0 + 8 * (c & 7) + (c >> 3) + 4 * n;
                                if (k > pos || k <= from) x[c] = 0xff800000u;
                            }
                        }
                    };
                    uint32_t x[32];
                    half(x, 0);
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 32; c += 2)
                        top = fmaxf(top, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
                    half(x, 1);
#pragma unroll
                    for (int c = 0; c < 32; c += 2)
                        top = fmaxf(top, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
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
                    float2 l2 = make_float2(0.0f, 0.0f);
                    uint32_t p[32];
#pragma unroll
                    for (int n = 1; n >= 0; n--) {
                        if (n == 0) half(x, 0);
                        if (far) {
#pragma unroll
                            for (int c = 0; c < 32; c++)
                                x[c] = __float_as_uint(__fmul_rn(__uint_as_float(x[c]), fs));
                        }
#pragma unroll
                        for (int c = 0; c < 16; c++) {
                            float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]),
                                                              __uint_as_float(x[2 * c + 1])), f2, s2);
                            e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                            l2 = __fadd2_rn(l2, e);
                            p[16 * n + c] = F16::pack(e.x, e.y);
                        }
                    }
                    l += l2.x + l2.y;
                    __syncwarp();
                    tmem_store32(ts, p);
                    tc_wait_store();
                    any = true;
                }
                turns++;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[grp][buf]);
            }
            if (any) {  // the last step's P V
                waited(a, sh, &sh.o_done[grp], (turns - 1) & 1);
                tc_fence_after();
            }
        } else if (run && (grp == 2 || grp == 3)) {
            // ================= tiles of f16 values from the records: K, V^T =================
            const int t = tid & 127;
            const bool keys = grp == 2;
            const int seen = first_seen(a, s);
            while (true) {
                const uint32_t slot = steps % kNS, ks = steps % kNK, vs = vsteps % kNV;
                if (!waited(a, sh, &sh.rec_full[slot], (steps / kNS) & 1)) break;
                if (keys) {
                    if (steps >= kNK && !waited(a, sh, &sh.k_free[ks], (steps / kNK - 1) & 1)) break;
                } else {
                    if (vsteps >= kNV && !waited(a, sh, &sh.v_free[vs], (vsteps / kNV - 1) & 1)) break;
                }
                const int j = *reinterpret_cast<volatile int *>(&sh.info[steps % kInfo]);
                steps++;
                if (j >= 0) {
                    if (keys) form_k(sh.rec[slot], sh.k[ks], t);
                    else form_v(sh.rec[slot] + kRec, sh.v[vs], t, seen - 64 * j, s.n - 64 * j);
                    fence_proxy_async();
                }
                __syncwarp();
                if (lane == 0) {
                    if (keys) mbar_arrive(&sh.k_full[ks]);  // at the end too: it is a step
                    else if (j >= 0) mbar_arrive(&sh.v_full[vs]);
                    mbar_arrive(&sh.rec_free[slot]);
                }
                if (j < 0) break;
                vsteps++;
            }
        } else if (run && (warp == 16 || warp == 17)) {
            // ================= matrix instructions =================
            // One warp a tile. The whole warp goes through the steps, so that operand addresses stay
            // warp-uniform; one lane issues.
            const int g = warp - 16;
            const bool live = g == 0 || two, issuer = elect_one();
            const uint32_t k0 = smem_u32(sh.k[0]), v0 = smem_u32(sh.v[0]);
            const uint32_t qd = tc_desc(smem_u32(sh.q[0]) + g * 32768);
            // The scores of the next step, two ahead of the values: their place was P's of two steps
            // ago. False at the segment's end, which the softmax group learns of in the same way.
            auto next_scores = [&]() {
                const uint32_t ks = steps % kNK, d = tmem + col_s(g, steps);
                if (!waited(a, sh, &sh.k_full[ks], (steps / kNK) & 1)) return false;
                tc_fence_after();
                const int j = *reinterpret_cast<volatile int *>(&sh.info[steps % kInfo]);
                const bool more = __any_sync(0xffffffffu, j >= 0);
                const uint32_t kd = tc_desc(k0 + ks * 16384);
                if (issuer) {
                    if (more && live) {
#pragma unroll
                        for (int i = 0; i < 8; i++)  // 16 channels each
                            tc_mma(d, qd + (i >> 2) * 1024 + (i & 3) * 2,
                                   kd + (i >> 2) * 512 + (i & 3) * 2, kIdescS, i > 0);
                    }
                    tc_commit(&sh.s_full[g][steps & 1]);
                }
                steps++;
                return more;
            };
            // K's tile of a step is free once its scores have been read, V's once P V is done: both are
            // known here, and a plain arrival costs less than a commit.
            uint32_t pstep = steps;  // the step whose values come next
            bool cur = next_scores(), nxt = cur && next_scores();
            bool add = false;
            while (cur) {
                const uint32_t vs = vsteps % kNV;
                if (!waited(a, sh, &sh.v_full[vs], (vsteps / kNV) & 1)) break;
                if (!waited(a, sh, &sh.p_full[g][pstep & 1], (pstep >> 1) & 1)) break;
                tc_fence_after();
                const uint32_t p = tmem + col_s(g, pstep), d = tmem + kColO + g * 128;
                const uint32_t vd = tc_desc(v0 + vs * 16384);
                if (issuer) {
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 4; i++)  // 16 tokens each
                            tc_mma_ta(d, p + 8 * i, vd + 2 * i, kIdescO, add || i > 0);
                    }
                    tc_commit(&sh.o_done[g]);
                    mbar_arrive(&sh.k_free[pstep % kNK]);
                }
                if (!waited(a, sh, &sh.o_done[g], turns & 1)) break;
                if (issuer) mbar_arrive(&sh.v_free[vs]);
                vsteps++;
                turns++;
                pstep++;
                add = true;
                const bool third = nxt && next_scores();
                cur = nxt;
                nxt = third;
            }
            if (issuer) mbar_arrive(&sh.k_free[pstep % kNK]);  // the end's step
        } else if (run && warp == 18) {
            // ================= copies of the pages' records =================
            const int32_t *bt = a.block_table + (int64_t)b * a.max_blocks;
            const uint8_t *keep =
                a.keep_in ? a.keep_in + ((int64_t)b * a.Hkv + h) * a.max_blocks : nullptr;
            auto look = [&](int j) {
                int p = -1;
                if (j < j1 && (!keep || __ldg(keep + j))) {
                    p = __ldg(bt + j);
                    if (p < 0 || p >= a.P) {
                        raise_error(a.err, FFD_ERRBIT_BOUNDS);
                        p = -1;
                    }
                }
                return p;
            };
            auto push = [&](int j, int page) {
                const uint32_t slot = steps % kNS;
                if (steps >= kNS && !waited(a, sh, &sh.rec_free[slot], (steps / kNS - 1) & 1)) return false;
                if (lane == 0) {
                    *reinterpret_cast<volatile int *>(&sh.info[steps % kInfo]) = j;
                    if (j >= 0) {
                        const int64_t from = ((int64_t)page * a.Hkv + h) * kRec;
                        mbar_arrive_expect_tx(&sh.rec_full[slot], 2 * kRec);
                        tma_load_1d(sh.rec[slot], a.k4 + from, kRec, &sh.rec_full[slot]);
                        tma_load_1d(sh.rec[slot] + kRec, a.v4 + from, kRec, &sh.rec_full[slot]);
                    } else {
                        mbar_arrive(&sh.rec_full[slot]);
                    }
                }
                steps++;
                return true;
            };
            int ahead = look(j0 + lane);
            bool fine = true;
            for (int jb = j0; jb < j1 && fine; jb += 32) {
                const int page = ahead;
                ahead = look(jb + 32 + lane);
                for (uint32_t todo = __ballot_sync(0xffffffffu, page >= 0); todo && fine;
                     todo &= todo - 1) {
                    const int k = __ffs(todo) - 1;
                    fine = push(jb + k, __shfl_sync(0xffffffffu, page, k));
                }
            }
            if (fine) push(-1, -1);
        }

        // ---- the segment's results
        // (a whole item's rows by way of the tile's queries, which are read no more, so that lines of
        // out are written whole)
        float *mine = records + (int64_t)(kSlots * cta + (begins ? 1 : 0)) * kRecord;
        if (grp < 2 && run && (grp == 0 || two)) {
            const uint32_t to = tmem + ((uint32_t)(warp & 3) << 21) + kColO + grp * 128;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            float *row = mine + grp * kTile + r;
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
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            w[k] = T::pack(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                           __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                        *reinterpret_cast<uint4 *>(stage + r * 256 + (((4 * c + e) ^ (r & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (have) {
#pragma unroll
                    for (int e = 0; e < 32; e++) row[(32 * c + e) * kRows] = __uint_as_float(o[e]);
                }
            }
            if (complete) {
                named_barrier_sync(1 + grp, kTile);
#pragma unroll 4
                for (int k = 0; k < 16; k++) {
                    const int q = 32 * (warp & 3) + 2 * k + (lane >> 4), c = lane & 15;
                    const int i = div_g(a, row0 + grp * kTile + q);
                    if (i < s.nq)
                        *reinterpret_cast<uint4 *>(
                            static_cast<uint16_t *>(a.out) +
                            ((int64_t)(s.t0 + i) * a.Hq + h * a.G + row0 + grp * kTile + q - i * a.G) *
                                kD + 8 * c) =
                            *reinterpret_cast<const uint4 *>(stage + q * 256 + ((c ^ (q & 7)) << 4));
                }
            }
            if (have) {
                if (!complete) row[128 * kRows] = m, row[129 * kRows] = l;
                else if (a.lse)
                    a.lse[(int64_t)(s.t0 + qi) * a.Hq + h * a.G + rr - qi * a.G] = lse_of(m - kShift, l);
            }
        }
        if (!complete) {
            // the last of the CTAs that share the item joins their records (of many: in two steps)
            const Shares p(first, np, ncta, total, cta, kOnce);
            __syncthreads();
            if (tid == 0) sh.flag = p.last_of_group(tickets);
            __syncthreads();
            const int used = rows < kRows ? rows : kRows;
            // join records rec(0) .. rec(n - 1): 32 rows (one a lane) and 8 channels at a time, the
            // loads of five records together
            auto join = [&](auto rec, int n, auto done) {
                for (int k = warp; k < 16 * ((used + 31) / 32); k += kCtaWarps) {
                    const int q = 32 * (k >> 4) + lane, ch = 8 * (k & 15);
                    float M = -INFINITY, ls = 0.0f, o[8] = {};
                    for (int i0 = 0; i0 < n; i0 += 5) {
                        float v[5][8], mn[5], ln[5];
#pragma unroll
                        for (int i = 0; i < 5; i++) {
                            const bool in = i0 + i < n;
                            const float *from = rec(in ? i0 + i : i0) + q;
#pragma unroll
                            for (int c = 0; c < 8; c++) v[i][c] = __ldcg(from + (ch + c) * kRows);
                            mn[i] = in ? __ldcg(from + 128 * kRows) : -INFINITY;
                            ln[i] = __ldcg(from + 129 * kRows);
                        }
                        float Mn = M;
#pragma unroll
                        for (int i = 0; i < 5; i++) Mn = fmaxf(Mn, mn[i]);
                        const float al = M == -INFINITY ? 0.0f : ex2_approx(M - Mn);
                        M = Mn;
                        ls *= al;
#pragma unroll
                        for (int c = 0; c < 8; c++) o[c] *= al;
#pragma unroll
                        for (int i = 0; i < 5; i++) {
                            if (mn[i] == -INFINITY) continue;  // nothing in it: o and l are 0
                            const float f = ex2_approx(mn[i] - M);
                            ls = fmaf(f, ln[i], ls);
#pragma unroll
                            for (int c = 0; c < 8; c++) o[c] = fmaf(f, v[i][c], o[c]);
                        }
                    }
                    if (q < used) done(q, ch, M, ls, o);
                }
            };
            auto finish = [&](int q, int ch, float M, float ls, const float (&o)[8]) {
                const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                const int i = div_g(a, row0 + q), head = h * a.G + row0 + q - i * a.G;
                const int64_t at_row = (int64_t)(s.t0 + i) * a.Hq + head;
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at_row * kD + ch) =
                    make_uint4(T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv),
                               T::pack(o[4] * inv, o[5] * inv), T::pack(o[6] * inv, o[7] * inv));
                if (a.lse && ch == 0) a.lse[at_row] = lse_of(M - kShift, ls);
            };
            auto slot = [&](int c, int n) { return records + (int64_t)(kSlots * c + n) * kRecord; };
            if (sh.flag) {
                // a CTA's record: its second one when the item begins there, else its first
                auto member = [&](int n) { return slot(p.g0 + n, p.g0 + n == p.p0); };
                if (p.groups == 1) {
                    join(member, p.members, finish);
                } else {
                    float *group = slot(p.g0, p.g0 == p.p0 ? 2 : 3);
                    join(member, p.members, [&](int q, int ch, float M, float ls, const float (&o)[8]) {
#pragma unroll
                        for (int c = 0; c < 8; c++) group[(ch + c) * kRows + q] = o[c];
                        if (ch == 0) group[128 * kRows + q] = M, group[129 * kRows + q] = ls;
                    });
                    __syncthreads();
                    if (tid == 0) sh.flag = p.last_group(tickets);
                    __syncthreads();
                    if (sh.flag)
                        join([&](int n) { return slot(p.p0 + n * p.size, n ? 3 : 2); }, p.groups, finish);
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();

        // ---- the next item
        x = first + at + cnt;
        into = 0;
        if (x < c1) {
            do {
                next_item();
                item_pages(a, s, rt, fp, np);
            } while (np == 0);
        }
    }
    if (stopped(sh)) {  // leave nothing in flight
        bool done = true;
        if (warp == 18 && lane == 0)
            for (uint32_t i = 0; i < kNS && i < steps; i++) {
                const uint32_t last = steps - 1 - i;
                done &= mbar_drain(&sh.rec_full[last % kNS], (last / kNS) & 1, drain_bound_ns(a.wait_ns));
            }
        if ((warp == 16 || warp == 17) && elect_one()) {
            tc_commit(&sh.drain[warp - 16]);
            done = mbar_drain(&sh.drain[warp - 16], 0, drain_bound_ns(a.wait_ns));
        }
        if (!done) raise_error(a.err, FFD_ERRBIT_TIMEOUT);
    }
    __syncthreads();
    __syncwarp();
    if (warp == 0) tmem_free(tmem, 512);
}

template <class T>
cudaError_t launch(const AttnArgs &a, const Plan &pl, cudaStream_t stream) {
    static int smem_set[kMaxDevicesTracked];
    constexpr int bytes = sizeof(Shared) + 1024;
    const cudaError_t e = raise_smem_limit(kv4_chunk_kernel<T>, bytes, smem_set);
    if (e != cudaSuccess) return e;
    char *ws = reinterpret_cast<char *>(a.err);
    kv4_chunk_kernel<T><<<pl.ctas, kThreads, bytes, stream>>>(
        a, reinterpret_cast<float *>(ws + pl.records), reinterpret_cast<int *>(ws + pl.tickets));
    return cudaGetLastError();
}

}  // namespace

int chunk_rows() { return kRows; }
int chunk_slots() { return kSlots; }
int chunk_once() { return kOnce; }
size_t chunk_record_bytes() { return kRecord * sizeof(float); }

cudaError_t launch_chunk(const AttnArgs &a, const Plan &pl, int dtype, cudaStream_t stream) {
    return dtype == FFD_DTYPE_BF16 ? launch<Bf16>(a, pl, stream) : launch<F16>(a, pl, stream);
}

}  // namespace kv4
}  // namespace ffd
