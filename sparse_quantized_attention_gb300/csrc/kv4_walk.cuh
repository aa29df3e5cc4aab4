// kv4_walk.cuh -- what the attention kernels over the 4-bit cache share: the sequences as a walk over
// their pages sees them, query scaling, and the forms that results are written in.
#pragma once

#include "kv4.cuh"
#include "ptx.cuh"

namespace ffd {
namespace kv4 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A column's (or row's) reference m is raised only when a score passes it by 2^kLazy: P, which carries
// 2^kShift at the reference, then reaches 2^15 and f16 holds it. That asks for kShift - m and m + kLazy to
// be exact to a fraction. Past kFar a reference is rounded by more than 2^-2, and from 2^24 (log2 units)
// on 7 - m may come out as 8 - m and m + 8 as m + 16: a score could stand 2^16 above m and not raise it. So
// there any larger score raises m (no product then passes it, and P is at most 2^8), and the products
// that the powers are taken of are rounded as m was. An infinite m belongs to a query with an infinity.
constexpr float kShift = 7.0f;
constexpr float kLazy = 8.0f;
constexpr float kFar = 4194304.0f;  // 2^22
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar && fabsf(m) < INFINITY; }

// One sequence as the walk sees it.
struct Seq {
    int n, t0, nq;  // tokens, first query row, query rows
    int fp, np;     // first page any query sees, pages from there to the last
};

// The first token that any query of the sequence sees.
__device__ __forceinline__ int first_seen(const AttnArgs &a, const Seq &s) {
    const int low = s.n - s.nq;
    return a.window > 0 && low >= a.window ? low - a.window + 1 : 0;
}

__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b, bool report) {
    Seq s;
    s.n = __ldg(a.seq_lens + b);
    const int cap = a.max_blocks * kPage;
    bool bad = s.n < 0 || s.n > cap;
    s.n = s.n < 0 ? 0 : (s.n > cap ? cap : s.n);
    s.t0 = b * a.max_q;
    s.nq = a.max_q;
    if (a.cu_q) {
        s.t0 = __ldg(a.cu_q + b);
        const int end = __ldg(a.cu_q + b + 1);
        if (s.t0 < 0 || end < s.t0 || end > a.total_q || end - s.t0 > a.max_q) {
            bad = true;
            s.nq = 0;
        } else {
            s.nq = end - s.t0;
        }
    }
    if (report && bad) raise_error(a.err, FFD_ERRBIT_BOUNDS);
    s.fp = first_seen(a, s) >> 6;
    s.np = s.n > 0 && s.nq > 0 ? ((s.n + kPage - 1) >> 6) - s.fp : 0;
    return s;
}

// A query enters the matrix instructions as f16 times the power of two that brings its largest
// magnitude `top` into [2^13, 2^14): mul; f takes scores of it to log2 units (sm log2(e) / mul).
__device__ __forceinline__ void query_scale(const AttnArgs &a, float top, float &mul, float &f) {
    int e = (int)(__float_as_uint(top) >> 23) - 127;
    e = e < -100 ? -100 : (e > 127 ? 127 : e);
    mul = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
    f = a.sm_scale * kLog2e * __uint_as_float((uint32_t)(127 + e - 13) << 23);
    f = fmaxf(f, 1.2e-38f);  // never 0: times -inf it has to stay -inf
}

// The CTAs that share a run of pages: items first .. first + np - 1 of `total`, cut into ncta equal
// ranges. CTAs p0 .. p1 have parts of it. Up to kOnce of them are joined at once; more in groups of
// about their number's root, then group by group, so that many CTAs read the records side by side.
// Three arrays of kMaxCtas tickets count who has come: to the group of p0 (or to all), to the groups
// that begin at a later CTA, and the groups that are joined. Each is indexed by a CTA in which at most
// one such run begins, or goes on from before.
struct Shares {
    int p0, p1, size, groups, g0, members;  // groups of `size`; this CTA's: its first CTA, its CTAs
    __device__ Shares(int first, int np, int ncta, int total, int cta, int once) {
        p0 = (int)(((int64_t)(first + 1) * ncta - 1) / total);
        p1 = (int)(((int64_t)(first + np) * ncta - 1) / total);
        const int n = p1 - p0 + 1;
        size = members = n;
        groups = 1;
        g0 = p0;
        if (n <= once) return;
        size = (int)ceilf(sqrtf((float)n));
        groups = (n + size - 1) / size;
        const int at = (cta - p0) / size * size;
        g0 = p0 + at;
        members = n - at < size ? n - at : size;
    }
    // One thread, after a barrier behind the CTA's writes. The last to come leaves the ticket at 0
    // for the next call.
    __device__ bool come(int *ticket, int of) const {
        const bool last = add_acq_rel_gpu(ticket, 1) == of - 1;
        if (last) *ticket = 0;
        return last;
    }
    __device__ bool last_of_group(int *tickets) const {
        return come(tickets + (g0 == p0 ? 0 : kMaxCtas) + g0, members);
    }
    __device__ bool last_group(int *tickets) const {
        return come(tickets + 2 * kMaxCtas + p0, groups);
    }
};

// Two channels of a row of out.
template <class T>
__device__ __forceinline__ void write_pair(const AttnArgs &a, int row, int hq, int ch, float x,
                                           float y) {
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) +
                                  ((int64_t)row * a.Hq + hq) * kD + ch) = T::pack(x, y);
}

// Log-sum-exp of a row: m the reference of l in log2 units.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace kv4
}  // namespace ffd
