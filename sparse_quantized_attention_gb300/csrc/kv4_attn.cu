// kv4_attn.cu -- softmax attention over the 4-bit cache (definition in ffd.h).
//
// One warp per (query row, head): the lanes hold four channels each, and the row's visible tokens
// are taken one by one with a running maximum and sum.
#include "kv4.cuh"

namespace ffd {
namespace kv4 {
namespace {

template <class T>
__global__ void __launch_bounds__(128) kv4_rows_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(item / a.Hq), hq = (int)(item - (int64_t)t * a.Hq);
    if (t >= a.total_q) return;
    int b, i;
    if (!row_of(a.cu_q, a.B, a.max_q, t, b, i)) {
        if (a.cu_q[b] < 0) raise_error(a.err, FFD_ERRBIT_BOUNDS);
        return;
    }
    int nq = a.max_q;
    if (a.cu_q) {
        const int end = a.cu_q[b + 1];
        nq = end - a.cu_q[b];
        if (end > a.total_q || nq > a.max_q) {
            raise_error(a.err, FFD_ERRBIT_BOUNDS);
            return;
        }
    }
    int n = a.seq_lens[b];
    const int cap = a.max_blocks * kPage;
    if (n < 0 || n > cap) {
        raise_error(a.err, FFD_ERRBIT_BOUNDS);
        n = n < 0 ? 0 : cap;
    }
    const int h = hq / a.G, pos = n - nq + i;
    const int first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    const uint2 qw = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) +
                                                      t * a.q_stride + hq * kD + 4 * lane);
    const float2 q0 = T::unpack(qw.x), q1 = T::unpack(qw.y);
    const int g = lane >> 3, word = (lane >> 1) & 3, half = lane & 1;
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int blk = first >> 6; blk <= (pos >> 6) && pos >= 0; blk++) {
        if (a.keep_in && !a.keep_in[((size_t)b * a.Hkv + h) * a.max_blocks + blk]) continue;
        const int page = a.block_table[(size_t)b * a.max_blocks + blk];
        if (page < 0 || page >= a.P) {
            raise_error(a.err, FFD_ERRBIT_BOUNDS);
            continue;
        }
        const int64_t rec = ((int64_t)page * a.Hkv + h) * kRec;
        for (int r = 0; r < kPage; r++) {
            const int j = blk * kPage + r;
            if (j < first || j > pos) continue;
            const int co = code_offset(r, g) + 4 * word, po = param_offset(r, g);
            __half2 kv[4], vv[4];
            decode_word(*reinterpret_cast<const uint32_t *>(a.k4 + rec + co),
                        *reinterpret_cast<const __half2 *>(a.k4 + rec + po), kv);
            decode_word(*reinterpret_cast<const uint32_t *>(a.v4 + rec + co),
                        *reinterpret_cast<const __half2 *>(a.v4 + rec + po), vv);
            const float2 k0 = __half22float2(half ? kv[2] : kv[0]);
            const float2 k1 = __half22float2(half ? kv[3] : kv[1]);
            const float2 v0 = __half22float2(half ? vv[2] : vv[0]);
            const float2 v1 = __half22float2(half ? vv[3] : vv[1]);
            const float s =
                a.sm_scale * warp_sum(q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y);
            const float mn = fmaxf(m, s);
            const float al = m == -INFINITY ? 0.0f : expf(m - mn);
            const float p = expf(s - mn);
            m = mn;
            l = l * al + p;
            o[0] = o[0] * al + p * v0.x;
            o[1] = o[1] * al + p * v0.y;
            o[2] = o[2] * al + p * v1.x;
            o[3] = o[3] * al + p * v1.y;
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const size_t row = (size_t)t * a.Hq + hq;
    uint2 w = make_uint2(T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv));
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * kD + 4 * lane) = w;
    if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_rows(const AttnArgs &a, int dtype, cudaStream_t stream) {
    const int64_t grid = ((int64_t)a.total_q * a.Hq + 3) / 4;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (dtype == FFD_DTYPE_BF16) kv4_rows_kernel<Bf16><<<(unsigned)grid, 128, 0, stream>>>(a);
    else kv4_rows_kernel<F16><<<(unsigned)grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace ffd
