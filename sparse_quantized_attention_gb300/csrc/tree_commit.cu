// tree_commit.cu -- the drafted path that the model confirms, found and moved into place
// (ffd_tree_commit in ffd.h).
//
// A block takes one sequence and KV head. Each thread owns a node: whether it is accepted and how deep it
// lies follow from doubling steps towards the root (eight at most), so that no block walks the tree.
// Every block of a sequence finds the path for itself (a few microseconds of latency; a second launch
// would cost as much) and moves its own head's rows: 32 rows are read, then written. A path's nodes
// ascend, node t of it at or behind place t, so what a later batch reads lies behind all that an earlier
// one has written.
//
// Latency is all it has: 3.4 us of a graph for one tree, 6.1 for 64 trees of 25 to 61 nodes with 8 heads (512
// blocks), which move 1.6 MB.
#include "tree.cuh"

namespace ffd {
namespace tree {
namespace {

constexpr int kThreads = 256;
static_assert(kThreads == kMaxNodes, "a thread a node");

struct Row {  // a token's place in the cache
    int page, row;
    bool ok;
};

__device__ __forceinline__ Row row_at(const CommitArgs &a, int b, int token) {
    Row r;
    r.page = __ldg(a.block_table + (int64_t)b * a.max_blocks + (token >> 6));
    r.row = token & 63;
    r.ok = r.page >= 0 && r.page < a.P;
    return r;
}

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const CommitArgs a) {
    __shared__ int up[2][kMaxNodes], deep[2][kMaxNodes], good[2][kMaxNodes];
    __shared__ int node[kMaxNodes];
    __shared__ int best;
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x - b * a.Hkv, i = threadIdx.x;
    const bool speaks = h == 0;  // writes the sequence's results and errors
    const int n = __ldg(a.seq_lens + b);
    int t0 = b * a.each, nq = a.each;
    bool bad = false;
    if (a.cu) {
        t0 = __ldg(a.cu + b);
        const int end = __ldg(a.cu + b + 1);
        bad = t0 < 0 || end < t0 || end > a.T;
        nq = bad ? 0 : end - t0;
    }
    const int rows = nq;  // of path
    if (n < nq || n > a.max_blocks * kPage || nq > kMaxNodes) bad = true, nq = 0;
    if (bad && speaks && i == 0) raise_error(a.err, FFD_ERRBIT_BOUNDS);
    if (nq == 0) {
        if (speaks) {
            for (int t = i; t < rows; t += kThreads) a.path[t0 + t] = -1;
            if (i == 0) a.accepted[b] = 0, a.next_token[b] = -1, a.new_lens[b] = n;
        }
        return;
    }
    // ---- parent, and whether the node fits behind it
    int p = -1, fits = 0;
    if (i < nq) {
        p = a.parents ? __ldg(a.parents + t0 + i) : i - 1;
        if (p < -1 || p >= i) {
            if (speaks) raise_error(a.err, FFD_ERRBIT_BOUNDS);
            p = -1;
        }
        fits = i == 0 || (p >= 0 && __ldg(a.draft + t0 + i) == __ldg(a.target + t0 + p));
    }
    if (i == 0) best = 0;
    up[0][i] = p;
    deep[0][i] = p >= 0;
    good[0][i] = fits;
    __syncthreads();
    // ---- all ancestors, by doubling
    int now = 0, d = p >= 0, g = fits, q = p;
    for (; __syncthreads_or(q >= 0); now ^= 1) {
        if (q >= 0) {
            d += deep[now][q];
            g &= good[now][q];
            q = up[now][q];
        }
        up[now ^ 1][i] = q;
        deep[now ^ 1][i] = d;
        good[now ^ 1][i] = g;
        __syncthreads();
    }
    // a chain's last node has 255 ancestors: depth above, then the lower index
    if (i < nq && g) atomicMax(&best, d << 8 | (kMaxNodes - 1 - i));
    __syncthreads();
    const int last = kMaxNodes - 1 - (best & (kMaxNodes - 1)), count = (best >> 8) + 1;
    // ---- the path: an accepted node is on it when it is the last one or one of its ancestors
    up[0][i] = p;
    __syncthreads();
    if (i == 0)
        for (int x = last, t = count - 1; t >= 0; t--, x = up[0][x]) node[t] = x;
    __syncthreads();
    if (speaks) {
        for (int t = i; t < nq; t += kThreads) a.path[t0 + t] = t < count ? node[t] : -1;
        if (i == 0) {
            a.accepted[b] = count;
            a.next_token[b] = __ldg(a.target + t0 + last);
            a.new_lens[b] = n - nq + count;
        }
    }
    // ---- rows, eight lanes each: 32 a batch
    const int lane = i & 7;
    for (int t = i >> 3; (t & ~31) < count; t += 32) {
        const bool moves = t < count && node[t] != t;
        Row from, to;
        bool go = false;
        uint4 x[2][2];
        uint4 r8;
        uint32_t r2 = 0, c4 = 0, p4 = 0;
        int64_t fk = 0, tk = 0;
        if (moves) {
            from = row_at(a, b, n - nq + node[t]);
            to = row_at(a, b, n - nq + t);
            go = from.ok && to.ok;
            if (!go && speaks && lane == 0) raise_error(a.err, FFD_ERRBIT_BOUNDS);
        }
        if (go) {
            fk = (int64_t)from.page * a.Hkv + h;
            tk = (int64_t)to.page * a.Hkv + h;
#pragma unroll
            for (int w = 0; w < 2; w++) {
                const uint8_t *src = w ? a.v : a.k;
                if (src) {
                    const uint4 *at = reinterpret_cast<const uint4 *>(src + (fk * kPage + from.row) * 256);
                    x[w][0] = at[lane];
                    x[w][1] = at[lane + 8];
                }
            }
            if (a.thumb) {  // codes 32 B, scales and zeros 8 B each; residual codes 128 B, scales 8 B
                const uint8_t *th = a.thumb + fk * kThumbRec, *re = a.resid + fk * kResidRec;
                c4 = reinterpret_cast<const uint32_t *>(th + from.row * kThumbRow)[lane];
                if (lane < 4)
                    p4 = reinterpret_cast<const uint32_t *>(
                        th + (lane < 2 ? kThumbScaleOff : kThumbZeroOff) + from.row * 8)[lane & 1];
                r8 = *reinterpret_cast<const uint4 *>(re + from.row * kD + 16 * (lane ^ (from.row & 7)));
                if (lane < 2)
                    r2 = reinterpret_cast<const uint32_t *>(re + kResidScaleOff + from.row * 8)[lane];
            }
        }
        __syncthreads();
        if (go) {
#pragma unroll
            for (int w = 0; w < 2; w++) {
                uint8_t *dst = w ? a.v : a.k;
                if (dst) {
                    uint4 *at = reinterpret_cast<uint4 *>(dst + (tk * kPage + to.row) * 256);
                    at[lane] = x[w][0];
                    at[lane + 8] = x[w][1];
                }
            }
            if (a.thumb) {
                uint8_t *th = a.thumb + tk * kThumbRec, *re = a.resid + tk * kResidRec;
                reinterpret_cast<uint32_t *>(th + to.row * kThumbRow)[lane] = c4;
                if (lane < 4)
                    reinterpret_cast<uint32_t *>(th + (lane < 2 ? kThumbScaleOff : kThumbZeroOff) +
                                                 to.row * 8)[lane & 1] = p4;
                *reinterpret_cast<uint4 *>(re + to.row * kD + 16 * (lane ^ (to.row & 7))) = r8;
                if (lane < 2)
                    reinterpret_cast<uint32_t *>(re + kResidScaleOff + to.row * 8)[lane] = r2;
            }
        }
    }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitArgs &a, cudaStream_t stream) {
    tree_commit_kernel<<<a.B * a.Hkv, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace tree
}  // namespace ffd
