// kv4.cuh -- the 4-bit cache's format on the device: record addresses, element types, argument
// bundles and the two directions of the arithmetic (format in ffd.h).
#pragma once

#include "common.cuh"

namespace ffd {
namespace kv4 {

constexpr int kRec = FFD_KV4_RECORD_BYTES;
constexpr int kParamOff = 4096;  // (scale, off) pairs behind the codes
static_assert(kRec == 5120, "record size");
constexpr int kMaxCtas = 1024;     // of an attention launch (one per SM at most)
// Pages' time that an item of the chunk kernel costs besides its pages (queries, first copies, results:
// 19000 to 20000 cycles, 2100 a page).
constexpr int kChunkLead = 9;
// Pages' time that cutting items costs a CTA of the chunk kernel (a second start, records, joins): when
// it takes one item, and when it takes several and has two of them cut.
constexpr int kJoinPages = 24, kJoinPagesSeveral = 39;
constexpr float kMaxInput = 16384.0f;  // |off| <= |min| + 16/15 range stays inside f16

// Byte offset, inside a record, of the 16 code bytes of group g (32 channels) of token r.
__host__ __device__ inline int code_offset(int r, int g) {
    const int line = r >> 1;
    const int sector = (2 * (r & 1) + (g >> 1)) ^ (line & 3);
    return line * 128 + sector * 32 + (g & 1) * 16;
}
// Byte offset of the (scale, off) pair of group g of token r.
__host__ __device__ inline int param_offset(int r, int g) { return kParamOff + 16 * r + 4 * g; }

// Element types of rows (FFD_DTYPE_*): two elements of a 32-bit word as floats and back.
struct Bf16 {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    // of pairs, each half for itself: the smaller, and the larger (NaN when one of them is)
    static __device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
        uint32_t r;
        asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    static __device__ __forceinline__ uint32_t max2_nan(uint32_t x, uint32_t y) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    // the f16 pair h, rounded to this type
    static __device__ __forceinline__ uint32_t from_half2(__half2 h) {
        const float2 f = __half22float2(h);
        return pack(f.x, f.y);
    }
};
struct F16 {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    // of pairs, each half for itself: the smaller, and the larger (NaN when one of them is)
    static __device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
        uint32_t r;
        asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    static __device__ __forceinline__ uint32_t max2_nan(uint32_t x, uint32_t y) {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    static __device__ __forceinline__ uint32_t from_half2(__half2 h) {
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// The pair of nibbles (i, i + 4) of a code word as the f16 pair (16 + c_i, 16 + c_i+4): the code in
// the top four mantissa bits (6..9 of each half) under exponent 2^4.
template <int i>
__device__ __forceinline__ __half2 code_pair(uint32_t w) {
    uint32_t x;
    if (i == 0) x = w << 6;
    if (i == 1) x = w << 2;
    if (i == 2) x = w >> 2;
    if (i == 3) x = w >> 6;
    // (x & mask) | exponent as one operation: two immediates would take two
    asm("lop3.b32 %0, %0, %1, %2, 0xea;" : "+r"(x) : "r"(0x03c003c0u), "r"(0x4c004c00u));
    return *reinterpret_cast<const __half2 *>(&x);
}

// Values of one code word's eight channels, channels 8J + 2i and 8J + 2i + 1 in v[i].
__device__ __forceinline__ void decode_word(uint32_t w, __half2 param, __half2 (&v)[4]) {
    const __half2 s = __low2half2(param), o = __high2half2(param);
    v[0] = __hfma2(code_pair<0>(w), s, o);
    v[1] = __hfma2(code_pair<1>(w), s, o);
    v[2] = __hfma2(code_pair<2>(w), s, o);
    v[3] = __hfma2(code_pair<3>(w), s, o);
}

// The level (16 .. 31) of x whose quotient by the scale lies next to the boundary between `lo` and
// lo + 1: by the side of b = fma(lo + 1/2, scale, off) that x lies on, the even one on it.
__device__ __forceinline__ float boundary_level(float x, float lo, float scale, float off) {
    const float b = __fmaf_rn(lo + 0.5f, scale, off);
    const bool odd = (static_cast<int>(lo) & 1) != 0;
    return (x > b || (x == b && odd)) ? lo + 1.0f : lo;
}

// Sequence of row t and the row's place in it, from the offsets cu [B+1] (or uniform rows per
// sequence when cu is null). False when the row belongs to nobody.
__device__ __forceinline__ bool row_of(const int32_t *cu, int B, int per, int t, int &b, int &i) {
    if (!cu) {
        b = t / per;
        i = t - b * per;
        return true;
    }
    int lo = 0, hi = B;  // the largest b in [0, B) with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid;
        else hi = mid;
    }
    b = lo;
    const int c = __ldg(cu + lo);
    i = t - c;
    return c >= 0 && c <= t && t < __ldg(cu + lo + 1);
}

// Arguments of a write or a read.
struct RowsArgs {
    int B, Hkv, P, max_blocks, T, per;
    const int32_t *cu, *positions, *block_table;
    int64_t k_stride, v_stride;  // elements
    int *err;
};

// Arguments of an attention call.
struct AttnArgs {
    int B, Hq, Hkv, G, P, max_blocks, max_q, total_q, window;
    int whole_items;  // chunk kernel: items are not cut if the lengths are even enough
    int lead;         // chunk kernel: pages' time that an item counts for besides its pages
    uint32_t over_g;  // ceil(2^32 / G), too large by less than G / 2^32 of it (G > 1)
    int64_t q_stride;
    float sm_scale;
    const void *q;
    const uint8_t *k4, *v4, *keep_in;
    const int32_t *seq_lens, *cu_q, *block_table;
    void *out;
    float *lse;
    int *err;  // the workspace: error word first
    uint64_t wait_ns;
};

// Launch shape and workspace of an attention call (byte offsets behind the error word).
struct Plan {
    int cols;  // query columns of the decode kernel (8, 16, 24 or 32), 0: the chunk kernel
    int ctas;
    int whole_items, lead;  // chunk kernel, as in AttnArgs
    size_t tickets, records, parked, total;
};

}  // namespace kv4
}  // namespace ffd
