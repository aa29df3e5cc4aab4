// rope.cu -- rotary positions on the way into the 16-bit cache and its records (ffd_rope_append in
// ffd.h).
//
// A warp takes one token and a run of its rows (heads of q, k and v in that order), eight lanes a row: a lane
// holds two pieces of 8 channels that are each other's partners (or hold neighbouring pairs), so a
// rotation needs no other lane. The token's 64 angles are computed once a warp, two a lane, and handed
// round by shuffles; a row then costs its loads, 24 operations of rotation a lane and its stores.
//
// Bound by memory: 32768 tokens of 32/8 heads (805 MB) in 121 us, 6.6 TB/s or 98 % of the measured copy rate; one
// token of 64 sequences takes 3.3 us of a graph, which is a launch and three reads one after another.
#include "kv4.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "tree.cuh"

namespace ffd {
namespace tree {
namespace {

using kv4::Bf16;
using kv4::F16;

constexpr int kWarps = 4;   // a block
constexpr int kBatch = 2;   // rows of a lane whose loads are under way together

// Cosine and sine of p f, p a whole number below 2^24. The product with 1 / 2 pi is held in two parts
// (f's own is exact to 2^-48), so that what is left after the whole turns are taken off is good to
// 1e-7 turns below 2^24 radians: single numbers would lose a digit of it for every digit of p.
__device__ __forceinline__ void turn(float f, int p, float &c, float &s) {
    constexpr float kHi = 0.159154943091895346f;
    constexpr float kLo = (float)(0.159154943091895346 - (double)kHi);
    const float hi = __fmul_rn(f, kHi);
    const float lo = __fmaf_rn(f, kLo, __fmaf_rn(f, kHi, -hi));
    const float x = (float)p;
    const float e = __fmul_rn(x, hi), rest = __fmaf_rn(x, hi, -e);
    const float t = __fadd_rn(__fsub_rn(e, rintf(e)), __fmaf_rn(x, lo, rest));
    sincospif(2.0f * t, &s, &c);
}

template <class T>
__device__ __forceinline__ uint4 turned(const uint4 &x, const uint4 &y, const float *c, const float *s,
                                        float sign) {  // x cos + sign y sin, eight channels
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 a = T::unpack(xs[i]), b = T::unpack(ys[i]);
        r[i] = T::pack(fmaf(sign * b.x, s[2 * i], a.x * c[2 * i]),
                       fmaf(sign * b.y, s[2 * i + 1], a.y * c[2 * i + 1]));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <class T>
__device__ __forceinline__ uint4 turned_pairs(const uint4 &x, const float *c, const float *s) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 a = T::unpack(xs[i]);
        r[i] = T::pack(fmaf(-a.y, s[i], a.x * c[i]), fmaf(a.x, s[i], a.y * c[i]));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// With records, five blocks an SM (96 registers, 8 bytes spilled): 32768 tokens of 32/8 heads take 172 us with what
// the compiler would use (125 registers, four blocks), 154 so, 172 with six; 126 is the floor.
template <class T, bool kRecords>
__global__ void __launch_bounds__(32 * kWarps, kRecords ? 5 : 1) rope_append_kernel(const RopeArgs a) {
    __shared__ uint4 stage[kRecords ? kWarps : 1][4 * kBatch][16];  // rotated keys, rows of 256 B
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane & 7;
    const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
    const int t = (int)(item / a.parts);
    if (t >= a.T) return;  // warp-uniform
    const int heads = a.Hq + 2 * a.Hkv;
    const int first = (int)(item - (int64_t)t * a.parts) * a.per;
    const int end = first + a.per < heads ? first + a.per : heads;
    int b, i;
    if (!row_of_warp(a.cu, a.B, a.each, t, lane, b, i)) return;
    const int start = __ldg(a.positions + b);
    if (start < 0) return;
    const int64_t token = (int64_t)start + i;
    const bool inside = token < (int64_t)a.max_blocks * kPage;
    int page = -1;
    if (inside) page = __ldg(a.block_table + (int64_t)b * a.max_blocks + (token >> 6));
    const bool stored = page >= 0 && page < a.P;
    if (!stored && end > a.Hq && lane == 0) raise_error(a.err, FFD_ERRBIT_BOUNDS);
    const int row = (int)(token & 63);

    // ---- the lane's eight angles: e < 8
    const int half = a.rot >> 1;
    float c[8], s[8];
    if (a.rot > 0 && first < a.Hq + a.Hkv) {
        int p = a.places ? __ldg(a.places + t) : (int)(token < kMaxPlace ? token : kMaxPlace);
        if (p < 0 || p >= kMaxPlace) {
            if (lane == 0) raise_error(a.err, FFD_ERRBIT_RANGE);
            p = 0;
        }
        float mc[2], ms[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int e = (lane >> 3) + 4 * k;
            const int pair = a.interleaved ? 4 * u + (e & 3) + 32 * (e >> 2) : 8 * u + e;
            mc[k] = a.scale, ms[k] = 0.0f;
            if (pair < half) {
                turn(__ldg(a.inv_freq + pair), p, mc[k], ms[k]);
                mc[k] *= a.scale;
                ms[k] *= a.scale;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            c[e] = __shfl_sync(0xffffffffu, mc[e >> 2], u + 8 * (e & 3));
            s[e] = __shfl_sync(0xffffffffu, ms[e >> 2], u + 8 * (e & 3));
        }
    }
    // the lane's two pieces (channels 8 piece ..), and whether each is rotated
    const int hc = half >> 3;
    int pa = u, pb = u + 8;
    bool ra = 8 * u < a.rot, rb = 8 * u + 64 < a.rot;
    if (!a.interleaved) {
        ra = rb = u < hc;
        pa = ra ? u : 2 * u;  // 2 hc + 2 (u - hc)
        pb = ra ? u + hc : 2 * u + 1;
    }

    for (int h0 = first; h0 < end; h0 += 4 * kBatch) {
        uint4 xa[kBatch], xb[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const int h = h0 + 4 * k + (lane >> 3);
            const uint16_t *from = nullptr;
            if (h < end) {
                if (h < a.Hq) from = a.q + (int64_t)t * a.q_stride + h * kD;
                else if (h < a.Hq + a.Hkv) from = a.k_new + (int64_t)t * a.k_stride + (h - a.Hq) * kD;
                else from = a.v_new + (int64_t)t * a.v_stride + (h - a.Hq - a.Hkv) * kD;
                xa[k] = *reinterpret_cast<const uint4 *>(from + 8 * pa);
                xb[k] = *reinterpret_cast<const uint4 *>(from + 8 * pb);
            }
        }
        if (kRecords) __syncwarp();  // the stage has been read
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const int h = h0 + 4 * k + (lane >> 3);
            if (h >= end) continue;
            const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
            uint4 ya = xa[k], yb = xb[k];
            if (!is_v) {
                if (a.interleaved) {
                    if (ra) ya = turned_pairs<T>(xa[k], c, s);
                    if (rb) yb = turned_pairs<T>(xb[k], c + 4, s + 4);
                } else if (ra) {
                    ya = turned<T>(xa[k], xb[k], c, s, -1.0f);
                    yb = turned<T>(xb[k], xa[k], c, s, 1.0f);
                }
            }
            uint16_t *to = nullptr;
            const int64_t at = (((int64_t)page * a.Hkv + (h - a.Hq - (is_v ? a.Hkv : 0))) * kPage + row) * kD;
            if (is_q) to = a.q_out + (int64_t)t * a.q_out_stride + h * kD;
            else if (stored) to = is_v ? a.v + at : a.k ? a.k + at : nullptr;
            if (to) {
                *reinterpret_cast<uint4 *>(to + 8 * pa) = ya;
                *reinterpret_cast<uint4 *>(to + 8 * pb) = yb;
            }
            if (kRecords && !is_q && !is_v) {
                stage[warp][4 * k + (lane >> 3)][pa] = ya;
                stage[warp][4 * k + (lane >> 3)][pb] = yb;
            }
        }
        if (kRecords) {  // a group of 32 channels of a staged key for each lane
            __syncwarp();
            const int h = h0 + (lane >> 2), g = lane & 3;
            if (stored && h >= a.Hq && h < a.Hq + a.Hkv && h < end) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint4 x = stage[warp][lane >> 2][4 * g + k];
                    w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
                }
                quant::GroupCodes o;
                quant::quantize_group(w, o);
                if (o.bad) raise_error(a.err, FFD_ERRBIT_RANGE);
                const int64_t tile = (int64_t)page * a.Hkv + h - a.Hq;
                quant::store_group(o, a.thumb + tile * kThumbRec, a.resid + tile * kResidRec, row, g);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(RopeArgs a, int dtype, cudaStream_t stream) {
    const int heads = a.Hq + 2 * a.Hkv;
    if (a.T == 0) return cudaSuccess;
    // Rows a warp takes: all of a token's, so that its angles are computed once, unless that leaves SMs
    // without warps. us in a graph with 8 rows a warp, all, and by this rule: one token of 28/4 heads 2.9 4.7 2.9;
    // of 64 sequences, 32/8 heads 3.3 5.8 3.3; 32768 tokens 135 121 121.
    const int64_t want = (int64_t)a.T * heads / (152 * 32);
    int per = want < heads ? (int)((want + 4 * kBatch - 1) / (4 * kBatch)) * 4 * kBatch : heads;
    if (per < 4 * kBatch) per = 4 * kBatch;
    a.per = per;
    a.parts = (heads + per - 1) / per;
    const int64_t blocks = ((int64_t)a.T * a.parts + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto run = [&](auto kernel) { kernel<<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a); };
    if (dtype == FFD_DTYPE_F16) run(rope_append_kernel<F16, false>);
    else if (a.thumb) run(rope_append_kernel<Bf16, true>);
    else run(rope_append_kernel<Bf16, false>);
    return cudaGetLastError();
}

}  // namespace tree
}  // namespace ffd
