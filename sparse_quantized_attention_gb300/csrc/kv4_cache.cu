// kv4_cache.cu -- writing rows into the 4-bit cache and reading them back (format in ffd.h).
#include "kv4.cuh"

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

// One thread per (row, KV head, tensor, group of 32 channels).
template <class T>
__global__ void __launch_bounds__(256) kv4_write_kernel(const RowsArgs a, const uint16_t *k,
                                                        const uint16_t *v, uint8_t *k4,
                                                        uint8_t *v4) {
    const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int g = (int)(item & 3);
    const bool is_v = (item >> 2) & 1;
    const int64_t th = item >> 3;
    const int t = (int)(th / a.Hkv), h = (int)(th - (int64_t)t * a.Hkv);
    if (t >= a.T) return;
    int page, r;
    bool bad;
    if (!place(a, t, page, r, bad)) {
        if (bad) raise_error(a.err, FFD_ERRBIT_BOUNDS);
        return;
    }
    const uint16_t *src = is_v ? v + t * a.v_stride : k + t * a.k_stride;
    const uint4 *row = reinterpret_cast<const uint4 *>(src + h * kD + g * 32);
    float x[32];
#pragma unroll
    for (int c = 0; c < 4; c++) {
        const uint4 u = __ldg(row + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 f = T::unpack(w[j]);
            x[8 * c + 2 * j] = f.x;
            x[8 * c + 2 * j + 1] = f.y;
        }
    }
    float lo = x[0], hi = x[0];
    bool range = false;
#pragma unroll
    for (int c = 0; c < 32; c++) {
        lo = fminf(lo, x[c]);
        hi = fmaxf(hi, x[c]);
        range |= !(fabsf(x[c]) <= kMaxInput);
    }
    if (range) raise_error(a.err, FFD_ERRBIT_RANGE);
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = __half2float(hs);
    const __half ho = __float2half_rn(__fmaf_rn(-16.0f, s, lo));
    const float o = __half2float(ho);
    const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;  // 0: every level clamps to 16
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        w[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; i++)
            w[j] |= level(x[8 * j + i], s, o, inv) << (4 * ((i >> 1) + 4 * (i & 1)));
    }
    uint8_t *rec = (is_v ? v4 : k4) + ((int64_t)page * a.Hkv + h) * kRec;
    *reinterpret_cast<uint4 *>(rec + code_offset(r, g)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<__half2 *>(rec + param_offset(r, g)) = __halves2half2(hs, ho);
}

// One thread per (row, KV head, word of 8 channels).
template <class T>
__global__ void __launch_bounds__(256) kv4_read_kernel(const RowsArgs a, const uint8_t *k4,
                                                       const uint8_t *v4, uint16_t *k,
                                                       uint16_t *v) {
    const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int J = (int)(item & 15);
    const int64_t th = item >> 4;
    const int t = (int)(th / a.Hkv), h = (int)(th - (int64_t)t * a.Hkv);
    if (t >= a.T) return;
    int page, r;
    bool bad;
    const bool ok = place(a, t, page, r, bad);
    if (!ok && !bad) return;
    if (bad) raise_error(a.err, FFD_ERRBIT_BOUNDS);
#pragma unroll
    for (int which = 0; which < 2; which++) {
        uint16_t *dst = which ? (v ? v + t * a.v_stride : nullptr)
                              : (k ? k + t * a.k_stride : nullptr);
        if (!dst) continue;
        uint4 o = make_uint4(0, 0, 0, 0);
        if (ok) {
            const uint8_t *rec = (which ? v4 : k4) + ((int64_t)page * a.Hkv + h) * kRec;
            const uint32_t w =
                __ldg(reinterpret_cast<const uint32_t *>(rec + code_offset(r, J >> 2)) + (J & 3));
            const uint32_t pw =
                __ldg(reinterpret_cast<const uint32_t *>(rec + param_offset(r, J >> 2)));
            __half2 val[4];
            decode_word(w, *reinterpret_cast<const __half2 *>(&pw), val);
            o = make_uint4(T::from_half2(val[0]), T::from_half2(val[1]), T::from_half2(val[2]),
                           T::from_half2(val[3]));
        }
        *reinterpret_cast<uint4 *>(dst + h * kD + 8 * J) = o;
    }
}

}  // namespace

cudaError_t launch_write(const RowsArgs &a, int dtype, const void *k, const void *v, uint8_t *k4,
                         uint8_t *v4, cudaStream_t stream) {
    const int64_t items = (int64_t)a.T * a.Hkv * 8;
    if (items == 0) return cudaSuccess;
    const int64_t grid = (items + 255) / 256;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto *kp = static_cast<const uint16_t *>(k), *vp = static_cast<const uint16_t *>(v);
    if (dtype == FFD_DTYPE_BF16)
        kv4_write_kernel<Bf16><<<(unsigned)grid, 256, 0, stream>>>(a, kp, vp, k4, v4);
    else
        kv4_write_kernel<F16><<<(unsigned)grid, 256, 0, stream>>>(a, kp, vp, k4, v4);
    return cudaGetLastError();
}

cudaError_t launch_read(const RowsArgs &a, int dtype, const uint8_t *k4, const uint8_t *v4, void *k,
                        void *v, cudaStream_t stream) {
    const int64_t items = (int64_t)a.T * a.Hkv * 16;
    if (items == 0) return cudaSuccess;
    const int64_t grid = (items + 255) / 256;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto *kp = static_cast<uint16_t *>(k), *vp = static_cast<uint16_t *>(v);
    if (dtype == FFD_DTYPE_BF16)
        kv4_read_kernel<Bf16><<<(unsigned)grid, 256, 0, stream>>>(a, k4, v4, kp, vp);
    else
        kv4_read_kernel<F16><<<(unsigned)grid, 256, 0, stream>>>(a, k4, v4, kp, vp);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace ffd
