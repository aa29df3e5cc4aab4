// tree_attn.cu -- attention of a tree of drafted tokens over the 16-bit cache (ffd_tree_attention in
// ffd.h).
//
// The plain kernel: a block for each (node, query head), its warps taking the pages in turn, a lane two
// keys of a page for the scores and four channels for the values.
#include "kv4.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace ffd {
namespace tree {
namespace {

constexpr int kWarps = 4;

template <class T>
__global__ void __launch_bounds__(32 * kWarps) tree_plain_kernel(const AttnArgs a) {
    __shared__ float q[kD];
    __shared__ uint32_t sees[kMaxNodes / 32];
    __shared__ int depth;
    __shared__ float of[kWarps][kD], ms[kWarps], ls[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, hq = blockIdx.y, h = hq / a.G;
    if (a.cu_q && t == 0 && hq == 0)  // offsets, wherever they lead
        for (int s = threadIdx.x; s < a.B; s += blockDim.x) {
            const int at = a.cu_q[s], end = a.cu_q[s + 1];
            if (at < 0 || end < at || end > a.total_q || end - at > a.max_q) raise_error(a.err, FFD_ERRBIT_BOUNDS);
        }
    int b, i;
    if (!row_of_warp(a.cu_q, a.B, a.max_q, t, lane, b, i)) return;
    int t0 = t - i, nq = a.max_q, n = a.seq_lens[b];
    if (a.cu_q) {
        const int end = a.cu_q[b + 1];
        nq = end - t0;
        if (end > a.total_q || nq > a.max_q) {
            raise_error(a.err, FFD_ERRBIT_BOUNDS);
            return;
        }
    }
    const int cap = a.max_blocks * kPage;
    if (n > cap || n < nq) raise_error(a.err, FFD_ERRBIT_BOUNDS);
    if (n > cap) n = cap;
    if (n < nq) n = 0;
    const int first = n - nq;
    if (threadIdx.x < kMaxNodes / 32) sees[threadIdx.x] = 0;
    q[threadIdx.x] = T::unpack(a.q[(int64_t)t * a.q_stride + hq * kD + threadIdx.x]).x;
    __syncthreads();
    if (threadIdx.x == 0) {
        depth = i;
        if (a.parents) {
            depth = 0;
            for (int x = i;;) {
                if (a.window == 0 || depth < a.window) sees[x >> 5] |= 1u << (x & 31);
                int p = a.parents[t0 + x];
                if (p < -1 || p >= x) {
                    raise_error(a.err, FFD_ERRBIT_BOUNDS);
                    p = -1;
                }
                if (p < 0) break;
                x = p;
                depth++;
            }
        }
    }
    __syncthreads();
    const int pos = first + depth;
    const int from = a.window > 0 ? pos - a.window : -1;
    auto seen = [&](int j) {
        if (j < first) return j > from;
        const int x = j - first;
        if (a.parents) return x < nq && ((sees[x >> 5] >> (x & 31)) & 1u) != 0;
        return x <= i && j > from;
    };
    float m = -INFINITY, l = 0.0f, o[4] = {};
    const int lowest = a.window > 0 && first >= a.window ? first - a.window + 1 : 0;
    for (int j = (lowest >> 6) + warp; n > 0 && j * kPage <= first + i; j += kWarps) {
        if (a.keep_in && !a.keep_in[((int64_t)b * a.Hkv + h) * a.max_blocks + j]) continue;
        const int page = a.block_table[(int64_t)b * a.max_blocks + j];
        if (page < 0 || page >= a.P) {
            raise_error(a.err, FFD_ERRBIT_BOUNDS);
            continue;
        }
        const int64_t at = ((int64_t)page * a.Hkv + h) * kPage * kD;
        float s[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int r = 32 * e + lane;
            s[e] = -INFINITY;
            if (seen(64 * j + r)) {
                float x = 0.0f;
                const uint4 *row = reinterpret_cast<const uint4 *>(a.k + at + r * kD);
                for (int c = 0; c < 16; c++) {
                    const uint4 w = row[c];
                    const float2 x0 = T::unpack(w.x), x1 = T::unpack(w.y), x2 = T::unpack(w.z),
                                 x3 = T::unpack(w.w);
                    const float *y = q + 8 * c;
                    x += y[0] * x0.x + y[1] * x0.y + y[2] * x1.x + y[3] * x1.y + y[4] * x2.x + y[5] * x2.y +
                         y[6] * x3.x + y[7] * x3.y;
                }
                s[e] = x * a.sm_scale;
            }
        }
        const float mn = fmaxf(m, warp_max(fmaxf(s[0], s[1])));
        if (mn == -INFINITY) continue;
        const float al = m == -INFINITY ? 0.0f : expf(m - mn);
        m = mn;
        l *= al;
        for (int c = 0; c < 4; c++) o[c] *= al;
        for (int r = 0; r < kPage; r++) {
            const float x = __shfl_sync(0xffffffffu, s[r >> 5], r & 31);
            if (x == -INFINITY) continue;  // not seen: its value may be anything
            const float p = expf(x - m);
            const uint2 w = *reinterpret_cast<const uint2 *>(a.v + at + r * kD + 4 * lane);
            const float2 v0 = T::unpack(w.x), v1 = T::unpack(w.y);
            l += p;
            o[0] += p * v0.x, o[1] += p * v0.y, o[2] += p * v1.x, o[3] += p * v1.y;
        }
    }
    for (int c = 0; c < 4; c++) of[warp][4 * lane + c] = o[c];
    if (lane == 0) ms[warp] = m, ls[warp] = l;
    __syncthreads();
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
    for (int w = 0; w < kWarps; w++) top = fmaxf(top, ms[w]);
    for (int w = 0; w < kWarps; w++) {
        if (ms[w] == -INFINITY) continue;
        const float f = expf(ms[w] - top);
        sum += f * ls[w];
        out += f * of[w][threadIdx.x];
    }
    const int64_t at = (int64_t)t * a.Hq + hq;
    a.out[at * kD + threadIdx.x] = (uint16_t)T::pack(sum == 0.0f ? 0.0f : out / sum, 0.0f);
    if (a.lse && threadIdx.x == 0) a.lse[at] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_tree_attention(const AttnArgs &a, const Plan &, int dtype, cudaStream_t stream) {
    const dim3 grid(a.total_q, a.Hq);
    if (dtype == FFD_DTYPE_BF16) tree_plain_kernel<kv4::Bf16><<<grid, 32 * kWarps, 0, stream>>>(a);
    else tree_plain_kernel<kv4::F16><<<grid, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace tree
}  // namespace ffd
