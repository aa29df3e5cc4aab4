// kv4_decode.cu -- attention over the 4-bit cache for few query rows: up to 8 NT (row, head) pairs
// share a KV head (NT = 1: one decode token of any GQA group; NT = 2 to 4: drafted tokens).
//
// The definition is the one of ffd.h. The pages of all (sequence, KV head) units, concatenated, are
// cut into equal contiguous ranges, one per CTA, and a range is walked in windows of kWindow pages: what
// its list has room for (a unit that goes on in the next window leaves its state in a carry record). The
// CTA lists the window's pages that a mask keeps, each warp takes an equal share of the list and
// walks it alone: it has room for one page's K record and one V record in shared memory, each refilled
// by a bulk copy as soon as it has been read, computes
//   S = K q^T   (16 tokens x 8 columns a matrix instruction, 8 of them over the 128 channels),
//   P = 2^(S - m) against a reference m of each column, raised when a score passes it by 2^8,
//   O^T += V^T P^T (16 channels x 8 columns, 8 of them over the 128 channels)
// with K and V formed in registers from the codes (one shift, one logical operation and one fused
// multiply-add a pair of values, exact by the format), and keeps m, the sum l and O^T in registers
// throughout; no barrier stands in the loop. At the end a CTA's warps join their states through
// shared memory, and the last CTA of a unit joins those of the CTAs (order fixed by page, so the
// result does not depend on arrival).
//
// P is rounded to f16 with 2^7 at the reference, so probabilities down to 2^-21 of it keep all 11
// bits (and down to 2^-31 some). The reference follows the maximum lazily, which saves the rescaling
// that a new maximum in any of a warp's columns would cost nearly every time. q enters as f16 scaled
// by a power of two per column (its largest magnitude in [2^13, 2^14)): exact for bf16 and f16 queries
// apart from elements below 2^-27 of the largest.
//
// What bounds it. A page of a head is 10 KB for 64 x 8 NT scores. With one column tile a long cache is
// read at 4.9 TB/s (4 x 131072 tokens, 28/4 heads: 68 to 69 us, 72 % of the measured copy rate; forming K and
// V takes most of the issue slots then, a matrix instruction 8 cycles of a scheduler's), a batch of 32
// sequences at 5.1 TB/s (86 us). A short cache waits instead: about 3.5 us until the first copy is asked
// for, 2 us for it, 4 to 5 us for the join of the warps, the records and the tickets (4096 tokens:
// 12 us, 32768: 23 us). With more column tiles eight warps are all that the registers allow, and their
// instructions wait on one another (0.3 issued a cycle of a scheduler): 24 rows behind a window of 4096
// take 40 us, 16 % of the copy rate.
#include "kv4_walk.cuh"

namespace ffd {
namespace kv4 {
namespace {

constexpr int kSlot = 2 * kRec;       // a warp's K record and V record
constexpr int kStride = 132;          // floats of a joined column: o[128], m, l, two unused
constexpr int kWindow = 2048;         // pages of a CTA's list
// Records of a CTA: of the unit that goes on from before, of the one that begins there; two carries
// between windows; of a group of CTAs whose first one this is, where the unit begins or goes on.
constexpr int kSlots = 6;
constexpr int kOnce = 16;             // records that one CTA joins at once

// Warps of a CTA: what their registers allow (128 a thread for one column tile, 168 for two, 251 for three,
// 255 for four; 44, 84, 0 and 280 bytes a thread are spilled all the same), and the 16-token tiles that a
// warp takes together: the more column tiles, the fewer tokens it needs for its matrix instructions not to
// wait on one another.
template <int NT>
constexpr int kWarpsOf = NT == 1 ? 16 : NT == 2 ? 12 : 8;
template <int NT>
constexpr int kTogether = NT == 1 ? 4 : NT <= 3 ? 2 : 1;

// A page of a range's list.
struct Entry {
    int rec;    // page * Hkv + h; -1: dropped, listed because it is its unit's first in the window
    int unit;   // b * Hkv + h
    int j;      // block of the sequence
    int first;  // the unit's first item
};

template <int NT>
struct Shared {
    static constexpr int W = kWarpsOf<NT>;
    // a warp's K record and V record, later its last state
    uint8_t ring[W][kSlot > 8 * NT * kStride * 4 ? kSlot : (8 * NT * kStride * 4 + 15) / 16 * 16];
    Entry list[kWindow];
    uint64_t full[W][2];
    // Up to 32 sequences: each warp's own table of them and of the items before them, so that a short
    // call's warps begin without a barrier. More: items before each thread's chunk of sequences.
    Seq seqs[W][32];
    int start[W][32];
    int pre[32 * W];
    int scan[W];
    int unit[W][2], first[W][2];      // of a warp's parked and of its last state (unit -1: none)
    int flag[2];
};
static_assert(sizeof(Shared<1>) + 128 <= 232448 && sizeof(Shared<2>) + 128 <= 232448 &&
                  sizeof(Shared<3>) + 128 <= 232448 && sizeof(Shared<4>) + 128 <= 232448,
              "shared memory per CTA");

// Softmax state of a warp: columns 2 tig, 2 tig + 1 of each 8-column tile (tig = lane % 4). m is the
// columns' reference (log2 units), the same in all lanes of a column; l sums this lane's rows;
// o[t][c] is channel 16 g + c (and 16 g + 8 + c) of the two columns (g = lane / 4).
template <int NT>
struct State {
    float m[NT][2], l[NT][2], o[NT][8][4];
    __device__ void clear() {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int c = 0; c < 8; c++) o[t][c][0] = o[t][c][1] = o[t][c][2] = o[t][c][3] = 0.0f;
        }
    }
    // l of the whole column in every lane
    __device__ void close() {
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], x);
    }
};

// A column's row of q, out and lse; false when the column has none.
__device__ __forceinline__ bool column(const AttnArgs &a, const Seq &s, int h, int c, int &row,
                                       int &hq, int &i) {
    i = c / a.G;
    row = s.t0 + i;
    hq = h * a.G + c - i * a.G;
    return i < s.nq;
}

// Query fragments of the NT tiles: column g of tile t, channels 32 tig .. 32 tig + 31, as f16 pairs
// of q 2^(13 - e) (e: exponent of the column's largest magnitude); fs[t][2]: log2-unit factors
// sm log2(e) 2^(e - 13) of columns 2 tig, 2 tig + 1.
template <int NT, class T>
__device__ __forceinline__ void load_queries(const AttnArgs &a, const Seq &s, int h, int lane,
                                             uint32_t (&qf)[NT][16], float (&fs)[NT][2]) {
    const int g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; t++) {
        int row, hq, i;
        const bool have = column(a, s, h, 8 * t + g, row, hq, i);
        const uint4 *src = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(a.q) + (int64_t)(have ? row : 0) * a.q_stride +
            (have ? hq : 0) * kD + 32 * tig);
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint4 u = have ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
            w[4 * j] = u.x;
            w[4 * j + 1] = u.y;
            w[4 * j + 2] = u.z;
            w[4 * j + 3] = u.w;
        }
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const float2 f = T::unpack(w[j]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float mul, f;
        query_scale(a, top, mul, f);
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const float2 v = T::unpack(w[j]);
            qf[t][j] = F16::pack(v.x * mul, v.y * mul);
        }
        fs[t][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
        fs[t][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
    }
}

// Scores of TT 16-token tiles of a page: x[t][tile] as in the matrix instruction's result (rows g,
// g + 8 of the tile, columns 2 tig, 2 tig + 1). K of a row: the lane holds group tig of rows g and
// g + 8 of a tile, 16 code bytes and one (scale, off) pair each; codes and par point at row g's of the
// first tile.
template <int NT, int TT>
__device__ __forceinline__ void tile_scores(const uint8_t *codes, const uint8_t *par,
                                            const uint32_t (&qf)[NT][16], float (&x)[NT][TT][4]) {
#pragma unroll
    for (int tile = 0; tile < TT; tile++) {
        const uint4 c0 = *reinterpret_cast<const uint4 *>(codes + tile * 1024);
        const uint4 c1 = *reinterpret_cast<const uint4 *>(codes + tile * 1024 + 512);
        const __half2 p0 = *reinterpret_cast<const __half2 *>(par + tile * 256);
        const __half2 p1 = *reinterpret_cast<const __half2 *>(par + tile * 256 + 128);
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int t = 0; t < NT; t++) x[t][tile][0] = x[t][tile][1] = x[t][tile][2] = x[t][tile][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            __half2 v0[4], v1[4];
            decode_word(w0[j], p0, v0);
            decode_word(w1[j], p1, v1);
            const uint32_t *r0 = reinterpret_cast<const uint32_t *>(v0);
            const uint32_t *r1 = reinterpret_cast<const uint32_t *>(v1);
#pragma unroll
            for (int t = 0; t < NT; t++) {
                mma_f16(x[t][tile], r0[0], r1[0], r0[1], r1[1], qf[t][4 * j], qf[t][4 * j + 1]);
                mma_f16(x[t][tile], r0[2], r1[2], r0[3], r1[3], qf[t][4 * j + 2], qf[t][4 * j + 3]);
            }
        }
    }
}

// O^T += V^T P^T over TT tiles. The lane holds words 2 g, 2 g + 1 of tokens 2 tig, 2 tig + 1 of a tile
// and of the two eight further on: codes[e] and par point at token 2 tig (+ e for the codes) of the
// first tile. In a page that some query does not see whole, tokens before `seen` and from n on, which none sees
// (positions in the sequence, as `at` is token 2 tig's), may hold anything and count as 0. A permutation of
// bytes puts two tokens' nibbles of one channel into one register's halves.
template <int NT, int TT>
__device__ __forceinline__ void tile_values(const uint8_t *const (&codes)[2], const uint8_t *par,
                                            const AttnArgs &a, const Seq &sq, bool open, int at,
                                            const uint32_t (&pf)[NT][TT][2], State<NT> &st) {
#pragma unroll
    for (int tile = 0; tile < TT; tile++) {
        // [half of the tile] token pairs 16 tile + 8 half + 2 tig, + 1
        uint32_t s[2], o[2];
        uint2 c[2][2];
#pragma unroll
        for (int hi = 0; hi < 2; hi++) {
            uint32_t q0 = *reinterpret_cast<const uint32_t *>(par + tile * 256 + hi * 128);
            uint32_t q1 = *reinterpret_cast<const uint32_t *>(par + tile * 256 + hi * 128 + 16);
            if (!open) {
                const int t = at + 16 * tile + 8 * hi, seen = first_seen(a, sq);
                q0 = t >= seen && t < sq.n ? q0 : 0u;
                q1 = t + 1 >= seen && t + 1 < sq.n ? q1 : 0u;
            }
            s[hi] = __byte_perm(q0, q1, 0x5410);
            o[hi] = __byte_perm(q0, q1, 0x7632);
#pragma unroll
            for (int e = 0; e < 2; e++)
                c[hi][e] = *reinterpret_cast<const uint2 *>(codes[e] + tile * 1024 + hi * 512);
        }
#pragma unroll
        for (int e = 0; e < 2; e++) {  // even channels of the words, then odd ones
            const uint32_t sel = e ? 0x7632 : 0x5410;
            uint32_t w[2][2];  // [word][half]
#pragma unroll
            for (int hi = 0; hi < 2; hi++) {
                w[0][hi] = __byte_perm(c[hi][0].x, c[hi][1].x, sel);
                w[1][hi] = __byte_perm(c[hi][0].y, c[hi][1].y, sel);
            }
            uint32_t f[4][4];  // [channel pair i][a0..a3]
#pragma unroll
            for (int word = 0; word < 2; word++)
#pragma unroll
                for (int hi = 0; hi < 2; hi++) {
                    const __half2 ss = *reinterpret_cast<const __half2 *>(&s[hi]);
                    const __half2 oo = *reinterpret_cast<const __half2 *>(&o[hi]);
                    const uint32_t ww = w[word][hi];
                    const __half2 r[4] = {__hfma2(code_pair<0>(ww), ss, oo),
                                          __hfma2(code_pair<1>(ww), ss, oo),
                                          __hfma2(code_pair<2>(ww), ss, oo),
                                          __hfma2(code_pair<3>(ww), ss, oo)};
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        f[i][2 * hi + word] = *reinterpret_cast<const uint32_t *>(&r[i]);
                }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int t = 0; t < NT; t++)
                    mma_f16(st.o[t][2 * i + e], f[i][0], f[i][1], f[i][2], f[i][3], pf[t][tile][0],
                            pf[t][tile][1]);
        }
    }
}

// A unit that one warp walked whole: its rows, straight from the registers.
template <int NT, class T>
__device__ __forceinline__ void write_direct(const AttnArgs &a, const Seq &s, int h, int lane,
                                             const State<NT> &st) {
    const int g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            int row, hq, i;
            if (!column(a, s, h, 8 * t + 2 * tig + e, row, hq, i)) continue;
            const float l = st.l[t][e], inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint32_t w[8];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                w[c] = T::pack(st.o[t][2 * c][e] * inv, st.o[t][2 * c + 1][e] * inv);
                w[4 + c] = T::pack(st.o[t][2 * c][2 + e] * inv, st.o[t][2 * c + 1][2 + e] * inv);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) +
                                                   ((int64_t)row * a.Hq + hq) * kD + 16 * g);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            if (a.lse && g == 0) a.lse[(int64_t)row * a.Hq + hq] = lse_of(st.m[t][e] - kShift, l);
        }
}

__device__ __forceinline__ float4 scaled(float4 v, float f) {
    return make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ float4 plus(float4 o, float f, float4 v) {
    return make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
}
template <class T>
__device__ __forceinline__ void write_four(const AttnArgs &a, int row, int hq, int ch, float4 v) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + ((int64_t)row * a.Hq + hq) * kD + ch) =
        make_uint2(T::pack(v.x, v.y), T::pack(v.z, v.w));
}

// A warp's state as 8 NT columns of kStride floats.
template <int NT>
__device__ __forceinline__ void park(float *rec, int lane, const State<NT> &st) {
    const int g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float *col = rec + (8 * t + 2 * tig + e) * kStride;
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                *reinterpret_cast<float2 *>(col + 16 * g + c) =
                    make_float2(st.o[t][c][e], st.o[t][c + 1][e]);
                *reinterpret_cast<float2 *>(col + 16 * g + 8 + c) =
                    make_float2(st.o[t][c][2 + e], st.o[t][c + 1][2 + e]);
            }
            if (g == 0) *reinterpret_cast<float2 *>(col + 128) = make_float2(st.m[t][e], st.l[t][e]);
        }
}

// Bounded wait of a warp for one of its copies; `dead` once a wait ran out.
__device__ __forceinline__ void wait_copy(const AttnArgs &a, uint64_t *bar, uint32_t parity,
                                          bool &dead) {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = globaltimer_ns();
    bool late = false;
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > a.wait_ns) {
            late = true;
            break;
        }
    }
    if (late) {
        raise_error(a.err, FFD_ERRBIT_TIMEOUT);
        dead = true;
    }
}

template <int NT, class T>
__global__ void __launch_bounds__(32 * kWarpsOf<NT>, 1)
    kv4_decode_kernel(const AttnArgs a, float *parked, float *records, int *tickets) {
    constexpr int W = kWarpsOf<NT>, kThreads = 32 * W, cols = 8 * NT;
    constexpr int kRecord = cols * kStride;
    extern __shared__ uint8_t raw[];
    Shared<NT> &sh = *reinterpret_cast<Shared<NT> *>(align_shared<128>(raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;

    if (lane < 2) {
        mbar_init(&sh.full[warp][lane], 1);
        sh.unit[warp][lane] = -1;
    }
    fence_barrier_init();

    // ---- items before each sequence, or before each chunk of them -----------------------------
    const bool few = a.B <= 32;
    const int chunk = few ? 1 : (a.B + kThreads - 1) / kThreads;
    int own = 0, total;
    bool empty = false;  // a sequence has queries and nothing for them to see
    auto scan = [&](int v) {  // sum over the lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    if (few) {
        Seq s = {0, 0, 0, 0, 0};
        if (lane < a.B) s = seq_of(a, lane, cta == 0 && warp == 0);
        own = s.np * a.Hkv;
        empty = s.np == 0 && s.nq > 0;
        const int inc = scan(own);
        sh.seqs[warp][lane] = s;
        sh.start[warp][lane] = inc - own;
        total = __shfl_sync(0xffffffffu, inc, 31);
        empty = __any_sync(0xffffffffu, empty);
    } else {
        for (int b = tid * chunk; b < (tid + 1) * chunk && b < a.B; b++) {
            const Seq s = seq_of(a, b, cta == 0);
            own += s.np * a.Hkv;
            empty |= s.np == 0 && s.nq > 0;
        }
        const int inc = scan(own);
        if (lane == 31) sh.scan[warp] = inc;
        empty = __syncthreads_or(empty);
        const int v = lane < W ? sh.scan[lane] : 0;
        const int up = scan(v);
        total = __shfl_sync(0xffffffffu, up, 31);
        sh.pre[tid] = __shfl_sync(0xffffffffu, up - v, warp) + inc - own;
        __syncthreads();
    }
    __syncwarp();
    auto seq = [&](int b) { return few ? sh.seqs[warp][b] : seq_of(a, b, false); };
    if (empty) {
        for (int u = cta * W + warp; u < a.B * a.Hkv; u += gridDim.x * W) {
            const int b = u / a.Hkv, h = u - b * a.Hkv;
            const Seq s = seq(b);
            if (s.np > 0) continue;
            for (int c = 0; c < cols; c++) {
                int row, hq, i;
                if (!column(a, s, h, c, row, hq, i)) break;
                write_pair<T>(a, row, hq, 4 * lane, 0.0f, 0.0f);
                write_pair<T>(a, row, hq, 4 * lane + 2, 0.0f, 0.0f);
                if (a.lse && lane == 0) a.lse[(int64_t)row * a.Hq + hq] = -INFINITY;
            }
        }
    }
    // the items are cut into equal ranges r0 .. r1 - 1, one per CTA
    const int ncta = total < (int)gridDim.x ? total : (int)gridDim.x;
    if (cta >= ncta) return;
    const int r0 = (int)((int64_t)total * cta / ncta), r1 = (int)((int64_t)total * (cta + 1) / ncta);
    // item x as an entry: its unit, its block, its record when the block is to be taken
    auto entry_of = [&](int x) {
        Entry e = {-1, 0, 0, 0};
        int b = 0, rem;
        if (few) {
#pragma unroll
            for (int step = 16; step > 0; step >>= 1)  // the last sequence that starts at or before x
                if (b + step < a.B && sh.start[warp][b + step] <= x) b += step;
            rem = x - sh.start[warp][b];
        } else {
            int lo = 0, hi = a.B < kThreads ? a.B : kThreads;
            while (hi - lo > 1) {  // the last chunk that starts at or before x
                const int mid = (lo + hi) >> 1;
                if (sh.pre[mid] <= x) lo = mid;
                else hi = mid;
            }
            b = lo * chunk;
            rem = x - sh.pre[lo];
        }
        Seq s = seq(b);
        while (rem >= s.np * a.Hkv) {
            rem -= s.np * a.Hkv;
            s = seq(++b);
        }
        const int h = rem / s.np, j = rem - h * s.np;
        e.unit = b * a.Hkv + h;
        e.j = s.fp + j;
        e.first = x - j;
        if (!a.keep_in || __ldg(a.keep_in + (int64_t)e.unit * a.max_blocks + e.j)) {
            const int page = __ldg(a.block_table + (int64_t)b * a.max_blocks + e.j);
            if (page < 0 || page >= a.P) raise_error(a.err, FFD_ERRBIT_BOUNDS);
            else e.rec = page * a.Hkv + h;
        }
        return e;
    };

    uint8_t *kbuf = sh.ring[warp], *vbuf = kbuf + kRec;
    // where this lane's parts of a tile's K and V stand (rows 16 tile + ...)
    const int g = lane >> 2, tig = lane & 3;
    const uint8_t *kcodes = kbuf + code_offset(g, tig), *kpar = kbuf + param_offset(g, tig);
    const uint8_t *const vcodes[2] = {vbuf + code_offset(2 * tig, g >> 1) + 8 * (g & 1),
                                      vbuf + code_offset(2 * tig + 1, g >> 1) + 8 * (g & 1)};
    const uint8_t *vpar = vbuf + param_offset(2 * tig, g >> 1);
    uint64_t *kfull = &sh.full[warp][0], *vfull = &sh.full[warp][1];
    uint32_t taken = 0;  // pages this warp has finished
    bool dead = false;
    // a range is walked in windows w0 .. w1 - 1 that fit the list; a unit that goes on in the next
    // window leaves its joined state in one of the CTA's two carry records
    for (int w0 = r0, turn = 0; w0 < r1; w0 += kWindow, turn ^= 1) {
        const int w1 = r1 - w0 < kWindow ? r1 : w0 + kWindow;

        // ---- the window's pages ---------------------------------------------------------------
        // A share of the list is the same number of entries, the odd ones with the first warps (so
        // that a short list reaches all schedulers).
        int count = w1 - w0, i0, i1;
        auto share = [&]() {
            const int each = count / W, odd = count - each * W;
            i0 = each * warp + (warp < odd ? warp : odd);
            i1 = i0 + each + (warp < odd);
        };
        if (!a.keep_in) {  // every page is listed: a warp lists its own share
            share();
            for (int i = i0 + lane; i < i1; i += 32) sh.list[i] = entry_of(w0 + i);
            __syncwarp();
        } else {  // the pages that the mask drops are left out
            count = 0;
            for (int x0 = w0; x0 < w1; x0 += kThreads) {
                const int x = x0 + tid;
                Entry e = {-1, 0, 0, 0};
                bool in = false;
                if (x < w1) {
                    e = entry_of(x);
                    in = e.rec >= 0 || x == e.first || x == w0;
                }
                const uint32_t bal = __ballot_sync(0xffffffffu, in);
                if (x0 != w0) __syncthreads();  // sh.scan is read no more
                if (lane == 0) sh.scan[warp] = __popc(bal);
                __syncthreads();
                int before = 0, all = 0;
#pragma unroll
                for (int w = 0; w < W; w++) {
                    const int v = sh.scan[w];
                    before += w < warp ? v : 0;
                    all += v;
                }
                if (in) sh.list[count + before + __popc(bal & ((1u << lane) - 1u))] = e;
                count += all;
            }
            __syncthreads();
            share();
        }
        if (w0 != r0) {  // the last window's states have been joined
            if (lane < 2) sh.unit[warp][lane] = -1;
            __syncwarp();
        }

        // ---- this warp's share ----------------------------------------------------------------
        auto next = [&](int i) {  // the next page to fetch from i on, i1 when there is none
            while (i < i1 && sh.list[i].rec < 0) i++;
            return i;
        };
        auto fetch = [&](const uint8_t *from, uint8_t *to, uint64_t *bar, int i) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, kRec);
                tma_load_1d(to, from + (int64_t)sh.list[i].rec * kRec, kRec, bar);
            }
        };
        const uint32_t was = taken;
        uint32_t kissued = taken, vissued = taken;  // copies asked for, all but this window's done
        if (w0 != r0) fence_proxy_async();  // the room held the last window's states
        {
            const int i = next(i0);
            if (i < i1 && !dead) {
                fetch(a.k4, kbuf, kfull, i);
                fetch(a.v4, vbuf, vfull, i);
                kissued++, vissued++;
            }
        }
        for (int i = i0; i < i1;) {
            // one unit's part of the share: entries i .. ie - 1
            const int unit = sh.list[i].unit, first = sh.list[i].first, start = i;
            const int b = unit / a.Hkv, h = unit - b * a.Hkv;
            const Seq s = seq(b);
            State<NT> st;
            uint32_t qf[NT][16];
            float fs[NT][2];
            load_queries<NT, T>(a, s, h, lane, qf, fs);
            st.clear();
            bool far = false;  // one of the warp's references is
            const int low = s.n - s.nq;  // position of the first query
            for (; i < i1; i++) {
                const Entry e = sh.list[i];
                if (e.unit != unit) break;
                if (e.rec < 0 || dead) continue;
                const int ni = next(i + 1);
                const int t0 = 64 * e.j;
                const bool open = t0 + 63 <= low && (a.window == 0 || t0 > s.n - 1 - a.window);
                wait_copy(a, kfull, taken & 1, dead);
                constexpr int TT = kTogether<NT>;
#pragma unroll 1
                for (int tile = 0; tile < 4; tile += TT) {
                    float sc[NT][TT][4];
                    tile_scores<NT, TT>(kcodes + tile * 1024, kpar + tile * 256, qf, sc);
                    if (tile + TT == 4) {
                        __syncwarp();
                        if (ni < i1 && !__any_sync(0xffffffffu, dead)) {
                            fetch(a.k4, kbuf, kfull, ni);
                            kissued++;
                        }
                    }
                    // ---- masks, maxima, probabilities (scores still want their factor fs)
                    if (!open) {
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int c = 0; c < 2; c++) {
                                const int pos = low + (8 * t + 2 * tig + c) / a.G;
                                const int from = a.window > 0 ? pos - a.window : -1;
#pragma unroll
                                for (int k = 0; k < TT; k++)
#pragma unroll
                                    for (int r = 0; r < 2; r++) {
                                        const int tok = t0 + 16 * (tile + k) + 8 * r + g;
                                        if (tok > pos || tok <= from) sc[t][k][2 * r + c] = -INFINITY;
                                    }
                            }
                    }
                    float mx[NT][2];
                    bool up = false;
                    const float lazy = far ? 0.0f : kLazy;
#pragma unroll
                    for (int t = 0; t < NT; t++)
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            float top = fmaxf(sc[t][0][c], sc[t][0][2 + c]);
#pragma unroll
                            for (int k = 1; k < TT; k++)
                                top = fmaxf(top, fmaxf(sc[t][k][c], sc[t][k][2 + c]));
                            mx[t][c] = top * fs[t][c];
                            up |= mx[t][c] > st.m[t][c] + lazy;
                        }
                    if (__any_sync(0xffffffffu, up)) {
                        bool any_far = false;
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int c = 0; c < 2; c++) {
                                float top = fmaxf(mx[t][c], st.m[t][c]);
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                                const float al =
                                    top == -INFINITY ? 0.0f : ex2_approx(st.m[t][c] - top);
                                st.m[t][c] = top;
                                any_far |= is_far(top);
                                st.l[t][c] *= al;
#pragma unroll
                                for (int k = 0; k < 8; k++) {
                                    st.o[t][k][c] *= al;
                                    st.o[t][k][2 + c] *= al;
                                }
                            }
                        far = __any_sync(0xffffffffu, any_far);
                    }
                    uint32_t pf[NT][TT][2];
#pragma unroll
                    for (int t = 0; t < NT; t++) {
                        float f[2], add[2];
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            f[c] = far ? 1.0f : fs[t][c];
                            add[c] = kShift - (st.m[t][c] == -INFINITY ? 0.0f : st.m[t][c]);
                        }
                        if (far) {
#pragma unroll
                            for (int k = 0; k < TT; k++)
#pragma unroll
                                for (int r = 0; r < 4; r++)
                                    sc[t][k][r] = __fmul_rn(sc[t][k][r], fs[t][r & 1]);
                        }
#pragma unroll
                        for (int k = 0; k < TT; k++)
#pragma unroll
                            for (int r = 0; r < 2; r++) {
                                const float p0 = ex2_approx(fmaf(sc[t][k][2 * r], f[0], add[0]));
                                const float p1 = ex2_approx(fmaf(sc[t][k][2 * r + 1], f[1], add[1]));
                                st.l[t][0] += p0;
                                st.l[t][1] += p1;
                                pf[t][k][r] = movmatrix_trans(F16::pack(p0, p1));
                            }
                    }
                    if (tile == 0) wait_copy(a, vfull, taken & 1, dead);
                    const uint8_t *const vc[2] = {vcodes[0] + tile * 1024, vcodes[1] + tile * 1024};
                    tile_values<NT, TT>(vc, vpar + tile * 256, a, s, open, t0 + 16 * tile + 2 * tig, pf, st);
                }
                dead = __any_sync(0xffffffffu, dead);
                if (ni < i1 && !dead) {
                    fetch(a.v4, vbuf, vfull, ni);
                    vissued++;
                }
                taken++;
            }
            st.close();
            // ---- the part is done: written out when it is all of its unit, else kept for the join
            const bool whole =
                a.keep_in ? first >= w0 && first + s.np <= w1 &&
                                (start > i0 || i0 == 0 || sh.list[i0 - 1].unit != unit) &&
                                (i < i1 || i1 == count || sh.list[i1].unit != unit)
                          : first >= w0 + i0 && first + s.np <= w0 + i1;
            if (whole) {
                write_direct<NT, T>(a, s, h, lane, st);
            } else {
                const int last = i == i1;  // else more units follow and the copies' room is in use
                __syncwarp();
                park<NT>(last ? reinterpret_cast<float *>(kbuf)
                              : parked + ((int64_t)cta * W + warp) * kRecord,
                         lane, st);
                if (lane == 0) {
                    sh.unit[warp][last] = unit;
                    sh.first[warp][last] = first;
                }
            }
        }
        if (dead) {  // leave no copy in flight
            bool done = true;
            if (kissued != was) done = mbar_drain(kfull, (kissued - 1) & 1, drain_bound_ns(a.wait_ns));
            if (vissued != was) done &= mbar_drain(vfull, (vissued - 1) & 1, drain_bound_ns(a.wait_ns));
            if (!done) raise_error(a.err, FFD_ERRBIT_TIMEOUT);
        }
        __syncthreads();

        // ---- join the warps' states of each unit, then the CTAs' ------------------------------
        // Lane i has entry i: warp i / 2, parked (even) or last (odd); `same` are the entries of its
        // unit. A warp takes a column of a unit at a time, four channels a lane.
        const int eu = lane < 2 * W ? sh.unit[lane >> 1][lane & 1] : -1;
        const int ef = lane < 2 * W ? sh.first[lane >> 1][lane & 1] : 0;
        const float *waiting = parked + (int64_t)cta * W * kRecord;
        auto last_state = [&](int w) { return reinterpret_cast<const float *>(sh.ring[w]); };
        const uint32_t same = __match_any_sync(0xffffffffu, eu);
        const uint32_t leads = __ballot_sync(0xffffffffu, eu >= 0 && __ffs(same) - 1 == lane);
        uint32_t units = leads;
        for (int k = 0; units; k++, units &= units - 1) {
            const int lead = __ffs(units) - 1;
            const int u = __shfl_sync(0xffffffffu, eu, lead);
            const int first = __shfl_sync(0xffffffffu, ef, lead);
            const uint32_t run = __shfl_sync(0xffffffffu, same, lead);
            const int b = u / a.Hkv, h = u - b * a.Hkv;
            const Seq s = seq(b);
            const bool carried = first < w0 && w0 > r0;            // from the window before
            const bool goes_on = first + s.np > w1 && w1 < r1;     // into the next one
            const bool begins = first >= r0, complete = begins && first + s.np <= r1;
            const float *carry = records + (int64_t)(kSlots * cta + 2 + (turn ^ 1)) * kRecord;
            float *mine = records + (int64_t)(kSlots * cta + (goes_on ? 2 + turn : begins)) * kRecord;
            // units begin at different warps, so that a CTA of many of them keeps all warps busy
            const int live = s.nq * a.G < cols ? s.nq * a.G : cols;
            for (int c = (warp + k * (W / 2)) % W; c < live; c += W) {
                const int ch = 4 * lane;
                float2 ml = make_float2(-INFINITY, 0.0f);
                if (eu == u && (lane & 1))
                    ml = *reinterpret_cast<const float2 *>(last_state(lane >> 1) + c * kStride + 128);
                if (eu == u && !(lane & 1))
                    ml = *reinterpret_cast<const float2 *>(waiting + (lane >> 1) * kRecord +
                                                           c * kStride + 128);
                float M = warp_max(ml.x);
                float2 cm = make_float2(-INFINITY, 0.0f);
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (carried) {
                    cm = *reinterpret_cast<const float2 *>(carry + c * kStride + 128);
                    o = *reinterpret_cast<const float4 *>(carry + c * kStride + ch);
                    M = fmaxf(M, cm.x);
                }
                const float cf = cm.x == -INFINITY ? 0.0f : ex2_approx(cm.x - M);
                const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - M);
                const float l = fmaf(cf, cm.y, warp_sum(f * ml.y));
                o = scaled(o, cf);
                for (uint32_t left = run & 0x55555555u; left; left &= left - 1) {
                    const int i = __ffs(left) - 1;
                    const float w = __shfl_sync(0xffffffffu, f, i);
                    o = plus(o, w, *reinterpret_cast<const float4 *>(waiting + (i >> 1) * kRecord +
                                                                     c * kStride + ch));
                }
                for (uint32_t left = run & 0xaaaaaaaau; left;) {
                    float4 v[4];
                    float w[4];
#pragma unroll
                    for (int n = 0; n < 4; n++) {  // four states' loads at a time
                        const int i = left ? __ffs(left) - 1 : 1;
                        w[n] = __shfl_sync(0xffffffffu, f, i);
                        if (!left) w[n] = 0.0f;
                        v[n] = *reinterpret_cast<const float4 *>(last_state(i >> 1) + c * kStride + ch);
                        if (!left) v[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        left &= left - 1;
                    }
#pragma unroll
                    for (int n = 0; n < 4; n++) o = plus(o, w[n], v[n]);
                }
                if (complete && !goes_on) {
                    int row, hq, i;
                    column(a, s, h, c, row, hq, i);
                    write_four<T>(a, row, hq, ch, scaled(o, l == 0.0f ? 0.0f : 1.0f / l));
                    if (a.lse && lane == 0) a.lse[(int64_t)row * a.Hq + hq] = lse_of(M - kShift, l);
                } else {
                    *reinterpret_cast<float4 *>(mine + c * kStride + ch) = o;
                    if (lane == 0)
                        *reinterpret_cast<float2 *>(mine + c * kStride + 128) = make_float2(M, l);
                }
            }
        }
        // Units that other CTAs share, the first and the last at most: the last CTA to come joins
        // their records (complete by the barrier and the ticket). One warp takes each ticket. Of more
        // than kOnce CTAs, groups of neighbours join first, and the last of the groups joins these.
        __syncthreads();
        uint32_t shared_units = 0;
        for (units = leads; units; units &= units - 1) {
            const int lead = __ffs(units) - 1;
            const int u = __shfl_sync(0xffffffffu, eu, lead);
            const int first = __shfl_sync(0xffffffffu, ef, lead);
            if (first >= r0) {  // it begins here: nobody else's when it ends here
                const int end = first + seq(u / a.Hkv).np;
                if (end <= r1 || w1 < r1) continue;
            } else if (w1 < r1 && first + seq(u / a.Hkv).np > w1) {
                continue;  // goes on in the next window
            }
            shared_units |= 1u << lead;
        }
        if (shared_units == 0) {
            __syncthreads();
            continue;
        }
        {
            const uint32_t mine = warp == 0 ? shared_units : warp == 1 ? shared_units & (shared_units - 1) : 0;
            if (mine) {
                const int lead = __ffs(mine) - 1;
                const int u = __shfl_sync(0xffffffffu, eu, lead);
                const int first = __shfl_sync(0xffffffffu, ef, lead);
                const Shares p(first, seq(u / a.Hkv).np, ncta, total, cta, kOnce);
                if (lane == 0) sh.flag[warp] = p.last_of_group(tickets);
            }
        }
        __syncthreads();
        for (int k = 0; shared_units; k++, shared_units &= shared_units - 1) {
            if (!sh.flag[k]) continue;
            const int lead = __ffs(shared_units) - 1;
            const int u = __shfl_sync(0xffffffffu, eu, lead);
            const int first = __shfl_sync(0xffffffffu, ef, lead);
            const int b = u / a.Hkv, h = u - b * a.Hkv;
            const Seq s = seq(b);
            const Shares p(first, s.np, ncta, total, cta, kOnce);
            const int live = s.nq * a.G < cols ? s.nq * a.G : cols;
            // Record i stands at from + i * step, and `skip` further from the second on: a CTA's own is
            // its second one when the unit begins there, else its first. Eight are joined a round, column
            // by column; of groups, the joined ones once more.
            const int64_t own = (int64_t)kSlots * kRecord;
            const bool at_start = p.g0 == p.p0;
            const float *from = records + p.g0 * own + (at_start ? kRecord : 0);
            int64_t step = own, skip = at_start ? -kRecord : 0;
            int n = p.members;
            for (bool last = p.groups == 1;; last = true) {
                auto rec = [&](int i) { return from + i * step + (i ? skip : 0); };
                for (int c = warp; c < live; c += W) {
                    float M = -INFINITY, l = 0.0f;
                    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int k0 = 0; k0 < n; k0 += 8) {
                        float2 ml = make_float2(-INFINITY, 0.0f);
                        if (lane < 8 && k0 + lane < n)
                            ml = __ldcg(reinterpret_cast<const float2 *>(rec(k0 + lane) + c * kStride +
                                                                         128));
                        float4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            v[i] = k0 + i < n ? __ldcg(reinterpret_cast<const float4 *>(
                                                    rec(k0 + i) + c * kStride + 4 * lane))
                                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        const float Mn = fmaxf(M, warp_max(ml.x));
                        const float al = M == -INFINITY ? 0.0f : ex2_approx(M - Mn);
                        const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - Mn);
                        M = Mn;
                        l = fmaf(al, l, warp_sum(f * ml.y));
                        o = scaled(o, al);
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            o = plus(o, __shfl_sync(0xffffffffu, f, i), v[i]);
                    }
                    if (last) {
                        int row, hq, i;
                        column(a, s, h, c, row, hq, i);
                        write_four<T>(a, row, hq, 4 * lane, scaled(o, l == 0.0f ? 0.0f : 1.0f / l));
                        if (a.lse && lane == 0) a.lse[(int64_t)row * a.Hq + hq] = lse_of(M - kShift, l);
                    } else {
                        float *col = records + p.g0 * own + (at_start ? 4 : 5) * kRecord + c * kStride;
                        *reinterpret_cast<float4 *>(col + 4 * lane) = o;
                        if (lane == 0) *reinterpret_cast<float2 *>(col + 128) = make_float2(M, l);
                    }
                }
                if (last) break;
                __syncthreads();
                if (tid == 0) sh.flag[k] = p.last_group(tickets);
                __syncthreads();
                if (!sh.flag[k]) break;
                from = records + p.p0 * own + 4 * kRecord;
                step = p.size * own;
                skip = kRecord;
                n = p.groups;
            }
        }
        __syncthreads();
    }
}

template <int NT, class T>
cudaError_t launch(const AttnArgs &a, const Plan &pl, cudaStream_t stream) {
    static int smem_set[kMaxDevicesTracked];
    constexpr int bytes = sizeof(Shared<NT>) + 128;
    const cudaError_t e = raise_smem_limit(kv4_decode_kernel<NT, T>, bytes, smem_set);
    if (e != cudaSuccess) return e;
    char *ws = reinterpret_cast<char *>(a.err);
    kv4_decode_kernel<NT, T><<<pl.ctas, 32 * kWarpsOf<NT>, bytes, stream>>>(
        a, reinterpret_cast<float *>(ws + pl.parked), reinterpret_cast<float *>(ws + pl.records),
        reinterpret_cast<int *>(ws + pl.tickets));
    return cudaGetLastError();
}

}  // namespace

size_t decode_record_bytes(int cols) { return (size_t)cols * kStride * sizeof(float); }
int decode_slots() { return kSlots; }
int decode_warps(int cols) {
    return cols == 8 ? kWarpsOf<1> : cols == 16 ? kWarpsOf<2> : cols == 24 ? kWarpsOf<3> : kWarpsOf<4>;
}

cudaError_t launch_decode(const AttnArgs &a, const Plan &pl, int dtype, cudaStream_t stream) {
    const bool bf16 = dtype == FFD_DTYPE_BF16;
    if (pl.cols == 8) return bf16 ? launch<1, Bf16>(a, pl, stream) : launch<1, F16>(a, pl, stream);
    if (pl.cols == 16) return bf16 ? launch<2, Bf16>(a, pl, stream) : launch<2, F16>(a, pl, stream);
    if (pl.cols == 24) return bf16 ? launch<3, Bf16>(a, pl, stream) : launch<3, F16>(a, pl, stream);
    return bf16 ? launch<4, Bf16>(a, pl, stream) : launch<4, F16>(a, pl, stream);
}

}  // namespace kv4
}  // namespace ffd
