// kv4_cache.cu -- writing rows into the 4-bit cache and reading them back (format in ffd.h).
#include "kv4.cuh"
#include "ptx.cuh"

namespace ffd {
namespace kv4 {
namespace {

// Token index and page of row t; false when the row is to be skipped. `bad`: it named a token or a
// page out of range.
__device__ __forceinline__ bool place(const RowsArgs &a, int t, int &page, int &r, bool &bad) {
    int b, i;
    bad = false;
    if (!row_of(a.cu, a.B, a.per, t, b, i)) return false;
    const int p0 = __ldg(a.positions + b);
    if (p0 < 0) return false;
    const int64_t p = (int64_t)p0 + i;
    if (p >= (int64_t)a.max_blocks * kPage) {
        bad = true;
        return false;
    }
    page = __ldg(a.block_table + (size_t)b * a.max_blocks + (p >> 6));
    r = (int)(p & 63);
    bad = page < 0 || page >= a.P;
    return !bad;
}

// Code word of eight values: w[i] holds values 2 i and 2 i + 1, nibbles i and i + 4. With inv15 =
// 1 / (15 scale), y = sat((x - off) inv15 - 16 / 15) is the clamped code / 15, off by less than 7e-7 (four
// roundings of 2^-24 on a product below 2.1, two on the sum); 15 y is rounded by adding 1.5 * 2^23.
// Where one of the eight lies within 2e-5 of a boundary (15 * 7e-7 = 1.1e-5) it is decided by the side
// of the boundary that x lies on. Codes are put together as numbers of 16 bits.
template <class T>
__device__ __forceinline__ uint32_t encode_word(const uint32_t *w, float s, float o, float inv15) {
    constexpr float kRound = 12582912.0f;
    const float2 round = make_float2(kRound, kRound), back = make_float2(-kRound, -kRound);
    const float2 no = make_float2(-o, -o), fifteen = make_float2(15.0f, 15.0f);
    float2 y[4], r[4];
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 d = __fadd2_rn(T::unpack(w[i]), no);
        y[i] = make_float2(fma_sat(d.x, inv15, -16.0f / 15.0f), fma_sat(d.y, inv15, -16.0f / 15.0f));
        r[i] = __fadd2_rn(__ffma2_rn(y[i], fifteen, round), back);
        const float2 e = __ffma2_rn(y[i], fifteen, make_float2(-r[i].x, -r[i].y));
        off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
    }
    if (off > 0.5f - 2e-5f) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 x = T::unpack(w[i]);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float t = 15.0f * (e ? y[i].y : y[i].x), lo = floorf(t);
                if (fabsf(t - lo - 0.5f) < 2e-5f)
                    (e ? r[i].y : r[i].x) = boundary_level(e ? x.y : x.x, lo + 16.0f, s, o) - 16.0f;
            }
        }
    }
    float2 h = __ffma2_rn(r[1], make_float2(16.0f, 16.0f), r[0]);
    h = __ffma2_rn(r[2], make_float2(256.0f, 256.0f), h);
    h = __ffma2_rn(r[3], make_float2(4096.0f, 4096.0f), h);
    h = __fadd2_rn(h, round);  // the low 16 bits are the number
    return __byte_perm(__float_as_uint(h.x), __float_as_uint(h.y), 0x5410);
}

// Writing: a block takes 32 rows of one KV head, a thread one group of 32 channels of K or of V: its
// least and largest value need no other thread. The eight threads of a row sit together and rows
// follow one another, so a prompt's records are written in whole lines.
//
// What has to move is 256 B of a tensor's row in and 80 B out: 26 us for 32768 tokens of 8 heads, which take
// 36. No unit is full (54 % of DRAM's rate, 69 % of the issue slots, at about 10.5 thread instructions a
// value): a thread loads, waits, codes and ends, with half the warps resident. So the least and largest
// are taken of packed pairs, sums and products of coding are packed too, the clamp is a product's saturation,
// and values are unpacked again where they are coded, which keeps to 48 registers and five blocks an
// SM (40 registers, six blocks: spills, 4 % slower).
template <class T, bool kWide>
__global__ void __launch_bounds__(256) kv4_write_kernel(const RowsArgs a, const uint16_t *k,
                                                        const uint16_t *v, uint8_t *k4,
                                                        uint8_t *v4) {
    const int g = threadIdx.x & 3;
    const bool is_v = (threadIdx.x >> 2) & 1;
    const int t = blockIdx.x * 32 + (threadIdx.x >> 3), h = blockIdx.y;
    if (t >= a.T) return;
    const uint16_t *row = (is_v ? v + t * a.v_stride : k + t * a.k_stride) + h * kD + g * 32;
    uint32_t w[16];
    if (kWide) {
        load_32b(row, reinterpret_cast<uint32_t(&)[8]>(w[0]));
        load_32b(row + 16, reinterpret_cast<uint32_t(&)[8]>(w[8]));
    } else {
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row) + c);
            w[4 * c] = u.x;
            w[4 * c + 1] = u.y;
            w[4 * c + 2] = u.z;
            w[4 * c + 3] = u.w;
        }
    }
    int page, r;
    bool bad;
    if (!place(a, t, page, r, bad)) {
        if (bad) raise_error(a.err, FFD_ERRBIT_BOUNDS);
        return;
    }
    uint32_t least = w[0], most = w[0];
#pragma unroll
    for (int j = 1; j < 16; j++) {
        least = T::min2(least, w[j]);
        most = T::max2_nan(most, w[j]);
    }
    const float2 l2 = T::unpack(least), m2 = T::unpack(most);
    float lo = fminf(l2.x, l2.y), hi = max_nan(m2.x, m2.y);
    if (!(lo >= -kMaxInput && hi <= kMaxInput)) {
        // the group holds finite values all the same (a NaN codes as the least): attention multiplies
        // them by 0 in the rows that do not see the token
        raise_error(a.err, FFD_ERRBIT_RANGE);
        lo = fminf(fmaxf(lo, -kMaxInput), kMaxInput);
        hi = fmaxf(fminf(hi, kMaxInput), -kMaxInput);
    }
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = __half2float(hs);
    const __half ho = __float2half_rn(__fmaf_rn(-16.0f, s, lo));
    const float o = __half2float(ho);
    const float inv15 = s > 0.0f ? __frcp_rn(s) * (1.0f / 15.0f) : 0.0f;  // 0: every code is 0
    uint8_t *rec = (is_v ? v4 : k4) + ((int64_t)page * a.Hkv + h) * kRec;
    *reinterpret_cast<uint4 *>(rec + code_offset(r, g)) =
        make_uint4(encode_word<T>(w, s, o, inv15), encode_word<T>(w + 4, s, o, inv15),
                   encode_word<T>(w + 8, s, o, inv15), encode_word<T>(w + 12, s, o, inv15));
    *reinterpret_cast<__half2 *>(rec + param_offset(r, g)) = __halves2half2(hs, ho);
}

// Reading: a block takes 64 rows of one KV head, a thread sixteen channels of two rows (32 apart), of
// K and of V: four loads in flight a thread, and eight threads write a row's 256 B. Bound by memory:
// four sequences of 131072 tokens, 4 heads, in 216 us, 6.5 TB/s or 96 % of the measured copy rate.
constexpr int kReadRows = 64;
template <class T, bool kWide>
__global__ void __launch_bounds__(256) kv4_read_kernel(const RowsArgs a, const uint8_t *k4,
                                                       const uint8_t *v4, uint16_t *k,
                                                       uint16_t *v) {
    const int c = threadIdx.x & 7, h = blockIdx.y;  // channels 16 c .. 16 c + 15
    int t[2];
    bool ok[2], mine[2];
    uint2 code[2][2];
    uint32_t par[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        t[i] = blockIdx.x * kReadRows + 32 * i + (threadIdx.x >> 3);
        int page = 0, r = 0;
        bool bad = false;
        ok[i] = t[i] < a.T && place(a, t[i], page, r, bad);
        mine[i] = ok[i] || bad;
        if (bad) raise_error(a.err, FFD_ERRBIT_BOUNDS);
        const int64_t at = ((int64_t)page * a.Hkv + h) * kRec;
        const int co = code_offset(r, c >> 1) + 8 * (c & 1), po = param_offset(r, c >> 1);
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const uint8_t *rec = (w ? v4 : k4) + at;
            const bool want = ok[i] && (w ? v != nullptr : k != nullptr);
            code[i][w] = want ? __ldg(reinterpret_cast<const uint2 *>(rec + co)) : make_uint2(0, 0);
            par[i][w] = want ? __ldg(reinterpret_cast<const uint32_t *>(rec + po)) : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (!mine[i]) continue;  // a page out of range: zeros
#pragma unroll
        for (int w = 0; w < 2; w++) {
            uint16_t *dst = w ? v : k;
            if (!dst) continue;
            dst += t[i] * (w ? a.v_stride : a.k_stride) + h * kD + 16 * c;
            const __half2 p = *reinterpret_cast<const __half2 *>(&par[i][w]);
            __half2 x[8];
            decode_word(code[i][w].x, p, reinterpret_cast<__half2(&)[4]>(x[0]));
            decode_word(code[i][w].y, p, reinterpret_cast<__half2(&)[4]>(x[4]));
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = T::from_half2(x[e]);
            if (kWide) {
                store_32b(dst, o);
            } else {
                reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
                reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

// Rows of 32-byte accesses: aligned base and stride (of the tensors that are there).
// 131072 tokens of 8 heads are written in 130 us with them (5.4 TB/s) and 144 us with 16-byte ones, read
// back in 110 us (6.4 TB/s) and 224 us: rows off the 32 bytes make two threads write each sector.
bool wide(const void *k, int64_t ks, const void *v, int64_t vs) {
    const bool kw = !k || ((reinterpret_cast<uintptr_t>(k) & 31) == 0 && ks % 16 == 0);
    const bool vw = !v || ((reinterpret_cast<uintptr_t>(v) & 31) == 0 && vs % 16 == 0);
    return kw && vw;
}

}  // namespace

cudaError_t launch_write(const RowsArgs &a, int dtype, const void *k, const void *v, uint8_t *k4,
                         uint8_t *v4, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    const dim3 grid((a.T + 31) / 32, a.Hkv);
    auto *kp = static_cast<const uint16_t *>(k), *vp = static_cast<const uint16_t *>(v);
    const bool w = wide(k, a.k_stride, v, a.v_stride);
    auto run = [&](auto kernel) { kernel<<<grid, 256, 0, stream>>>(a, kp, vp, k4, v4); };
    if (dtype == FFD_DTYPE_BF16) run(w ? kv4_write_kernel<Bf16, true> : kv4_write_kernel<Bf16, false>);
    else run(w ? kv4_write_kernel<F16, true> : kv4_write_kernel<F16, false>);
    return cudaGetLastError();
}

cudaError_t launch_read(const RowsArgs &a, int dtype, const uint8_t *k4, const uint8_t *v4, void *k,
                        void *v, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    const dim3 grid((a.T + kReadRows - 1) / kReadRows, a.Hkv);
    auto *kp = static_cast<uint16_t *>(k), *vp = static_cast<uint16_t *>(v);
    const bool w = wide(k, a.k_stride, v, a.v_stride);
    auto run = [&](auto kernel) { kernel<<<grid, 256, 0, stream>>>(a, k4, v4, kp, vp); };
    if (dtype == FFD_DTYPE_BF16) run(w ? kv4_read_kernel<Bf16, true> : kv4_read_kernel<Bf16, false>);
    else run(w ? kv4_read_kernel<F16, true> : kv4_read_kernel<F16, false>);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace ffd
