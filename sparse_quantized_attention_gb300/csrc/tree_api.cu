// tree_api.cu -- C entries of speculative decoding over the 16-bit cache (declared in include/ffd.h):
// argument checks, workspace planning and launches.
#include <math.h>

#include "kv4.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace ffd {
namespace tree {
cudaError_t launch_rope_append(RopeArgs a, int dtype, cudaStream_t stream);
cudaError_t launch_tree_commit(const CommitArgs &a, cudaStream_t stream);
cudaError_t launch_tree_attention(const AttnArgs &a, const Plan &pl, int dtype, cudaStream_t stream);
int tree_slots();
size_t tree_record_bytes(int tiles);
}  // namespace tree
}  // namespace ffd

using namespace ffd;
using namespace ffd::tree;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = 1 << 28;  // nodes of a sequence x G
constexpr int64_t kMaxUnits = 65535;   // (sequence, KV head) pairs of an attention call
// Pages of all items and what they count for besides, in int32: equal shares may end four pages a CTA behind them.
constexpr int64_t kMaxWalk = INT32_MAX - 4 * kv4::kMaxCtas;
constexpr int kTileRows = 128;         // smallest group of rows that walks the cache together

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Whether n bytes at p and m bytes at q share any.
bool overlap(const void *p, int64_t n, const void *q, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

// T rows of `heads` heads of 16-bit elements, `stride` elements from one to the next.
struct Rows {
    const void *p;
    int64_t T, stride, heads;
    int64_t width() const { return 2 * heads * kD; }  // bytes
    int64_t span() const {  // from the first row to the last (at most about 2^61)
        if (!p || T < 1) return 0;
        const int64_t most = ((int64_t)1 << 60) / T;
        return 2 * (T - 1) * (stride < most ? stride : most) + width();
    }
};

// Whether two lots of rows share any byte. Rows at one distance may lie between each other's, as those of a
// fused projection do; at different distances they may not.
bool overlap(const Rows &a, const Rows &b) {
    if (!overlap(a.p, a.span(), b.p, b.span())) return false;
    if (a.stride != b.stride || a.T != b.T) return true;
    const int64_t step = 2 * a.stride;
    const int64_t d = static_cast<const char *>(b.p) - static_cast<const char *>(a.p);
    const int64_t r = (d % step + step) % step, m = (r - d) / step;  // row i of a, i + m of b: r apart
    auto both = [&](int64_t x) { return x < a.T && -x < a.T; };
    return (r < a.width() && both(m)) || (r + b.width() > step && both(m - 1));
}

struct Bytes {
    const void *p;
    int64_t n;
};
bool overlap(const Bytes &a, const Bytes &b) { return a.p && b.p && overlap(a.p, a.n, b.p, b.n); }
bool overlap(const Rows &a, const Bytes &b) { return b.p && overlap(a.p, a.span(), b.p, b.n); }
template <size_t n, class X>
bool overlap_any(const Bytes (&a)[n], const X &x) {
    for (const Bytes &y : a)
        if (overlap(x, y)) return true;
    return false;
}
template <size_t n>
bool overlap_each_other(const Bytes (&a)[n]) {
    for (size_t i = 0; i < n; i++)
        for (size_t j = 0; j < i; j++)
            if (overlap(a[i], a[j])) return true;
    return false;
}

bool known(int32_t dtype) { return dtype == FFD_DTYPE_BF16 || dtype == FFD_DTYPE_F16; }

bool row_stride(int64_t stride, int64_t heads) { return stride >= heads * kD && stride % 8 == 0; }

ffd_status check_params(const ffd_tree_params *p) {
    if (!p) return FFD_ERR_INVALID_ARG;
    if (p->batch < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_pages < 1 ||
        p->max_blocks_per_seq < 1 || p->max_q_len < 1 || p->total_q < 1 || p->window < 0 ||
        p->num_splits < 0 || p->wait_limit_us < 0)
        return FFD_ERR_INVALID_ARG;
    if (!known(p->dtype)) return FFD_ERR_INVALID_ARG;
    if (p->num_q_heads % p->num_kv_heads != 0) return FFD_ERR_INVALID_ARG;
    if (!isfinite(p->sm_scale) || !(p->sm_scale > 0.0f)) return FFD_ERR_INVALID_ARG;
    if (p->q_stride != 0 && !row_stride(p->q_stride, p->num_q_heads)) return FFD_ERR_INVALID_ARG;
    if (p->head_dim != kD || p->page_size != kPage) return FFD_ERR_UNSUPPORTED;
    if (p->num_q_heads / p->num_kv_heads > kMaxG) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)p->batch * p->num_kv_heads > kMaxUnits) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)p->max_blocks_per_seq * kPage > INT32_MAX) return FFD_ERR_UNSUPPORTED;
    // the cache's rows, and the pages that groups of rows walk, are counted by int32
    if ((int64_t)p->num_pages * p->num_kv_heads > INT32_MAX / kPage) return FFD_ERR_UNSUPPORTED;
    const int64_t pages = (int64_t)p->batch * p->num_kv_heads * ((int64_t)p->max_blocks_per_seq + kItemPages);
    const int64_t rows = (int64_t)p->max_q_len * (p->num_q_heads / p->num_kv_heads);
    if (rows > kMaxRows || pages > kMaxWalk ||
        pages > kMaxWalk / (rows / 64 + 1))  // a tile has more than 64 rows
        return FFD_ERR_UNSUPPORTED;
    return FFD_OK;
}

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// A mask that every CTA reads through before it begins, to share the kept blocks out evenly; a larger one is cut
// as if all of its blocks were kept. us in a graph cut so and evenly, 8 nodes of 8 heads: 64 kept blocks of 16
// sequences of 4000 to 32768 tokens (64 KB of mask) 168 60, of 32 of 8000 to 65536 (256 KB) 273 118; 16 nodes over 96
// blocks of 4 x 131072, 4 heads 37.8 28.5. Where all keep as many anyway the counting costs: 200 blocks of 16 x
// 65536 (128 KB) 151 150, 128 of 32 x 131072 (512 KB) 210 215; one sequence of 4096 13.4 14.1.
// Counting also takes a lane of one warp for each sequence and one list of blocks for each (sequence, head), so
// batches past 32 and sequences of several groups of rows are cut by all their blocks: 64 kept of 4000 to 32768 tokens,
// 8 nodes of 8 heads, 31 sequences 107, 32 111, 33 301, 64 481; 16 such of 28/4 heads, 36 nodes 57, 37 nodes (two groups) 131; 96
// of 4 x 131072, 36 nodes 34.6, 37 53.4.
constexpr int64_t kMaskUnits = 256, kMaskBytes = 1 << 18;

// Workspace: [error word | two counters per CTA | records per CTA]. The counters, the only part that
// has to start at zero, have the same place and size whatever the parameters and are left at zero, so that
// calls of different shapes can share a workspace.
ffd_status make_plan(const ffd_tree_params *p, Plan *pl) {
    const ffd_status st = check_params(p);
    if (st != FFD_OK) return st;
    const int64_t nodes = kTileRows / (p->num_q_heads / p->num_kv_heads);  // of a tile
    // Two tiles share what is read, which pays wherever there are rows for both. us with tiles one by one and
    // two at a time: four sequences of 32768, 8 heads, 160 rows 157 127, 240 rows 178 133; 4096 rows over
    // 32768 637 416. With rows for one tile alone the second's warps and memory cost: 64 sequences of 4096, 4
    // rows 177 and 183.
    pl->tiles = p->max_q_len <= nodes ? 1 : 2;
    const int64_t groups = (p->max_q_len + pl->tiles * nodes - 1) / (pl->tiles * nodes);
    const int64_t items = (int64_t)p->batch * p->num_kv_heads * groups;
    const int sms = current_sm_count();
    int64_t ctas = p->num_splits;
    if (ctas == 0) {
        if (sms <= 0) return FFD_ERR_CUDA;
        int64_t most = p->max_blocks_per_seq;  // pages that an item sees at most
        if (p->window > 0) {
            const int64_t seen = ((int64_t)p->window + p->max_q_len) / kPage + 2;
            most = most < seen ? most : seen;
        }
        const int64_t each = share_pages((int)most);
        ctas = items * ((most + each - 1) / each);
    }
    if (sms > 0 && ctas > sms) ctas = sms;
    if (ctas > kv4::kMaxCtas) ctas = kv4::kMaxCtas;
    pl->ctas = (int)ctas;
    // Equal shares are worked out by that warp too. Past its 32 sequences and past four groups they would change little.
    // us without them and with: 8 nodes of 4 heads over 8192, 32 sequences 98 98 (33 take 102); one head of 8192, four groups
    // 23.1 21.2, five 22.5 20.0, sixteen 28.5 28.7; 8 heads of 32768, four 118 118, five 143 143, sixteen 408 408.
    pl->shares = p->batch <= 32 && groups <= 4 && items <= ctas ? (int)(ctas / items) : 0;
    pl->groups = (int)groups;
    pl->by_mask = p->batch <= 32 && groups == 1 && (int64_t)p->batch * p->num_kv_heads <= kMaskUnits &&
                  (int64_t)p->batch * p->num_kv_heads * p->max_blocks_per_seq <= kMaskBytes;
    size_t off = kAlign;
    pl->tickets = off;
    off = align_up(off + 2 * kv4::kMaxCtas * sizeof(int));
    pl->records = off;
    off = align_up(off + (size_t)tree_slots() * pl->ctas * tree_record_bytes(pl->tiles));
    pl->total = off;
    return FFD_OK;
}

}  // namespace

extern "C" {

ffd_status ffd_rope_append(const ffd_rope_params *params, const void *q, const void *k_new,
                           const void *v_new, const float *inv_freq, const int32_t *rope_positions,
                           const int32_t *cu_tokens, const int32_t *positions,
                           const int32_t *block_table, void *q_out, void *k, void *v, uint8_t *thumb,
                           uint8_t *resid, int32_t *error_word, void *stream) {
    if (!params || !positions || !block_table) return FFD_ERR_INVALID_ARG;
    const ffd_rope_params &p = *params;
    if (p.batch < 1 || p.num_q_heads < 0 || p.num_kv_heads < 1 || p.num_pages < 1 ||
        p.max_blocks_per_seq < 1 || p.total_tokens < 0 || !known(p.dtype))
        return FFD_ERR_INVALID_ARG;
    if (p.rot_dim < 0 || p.rot_dim > kD || p.rot_dim % 16 != 0 || (p.interleaved & ~1) ||
        !isfinite(p.rot_scale) || (p.rot_dim > 0 && !inv_freq))
        return FFD_ERR_INVALID_ARG;
    const int64_t T = p.total_tokens;
    if (!cu_tokens && T % p.batch != 0) return FFD_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) && T > 0) return FFD_ERR_INVALID_ARG;
    if (!v || (!k && !thumb) || (thumb == nullptr) != (resid == nullptr)) return FFD_ERR_INVALID_ARG;
    if (T > 0 && (!k_new || !v_new)) return FFD_ERR_INVALID_ARG;
    const bool queries = q && p.num_q_heads > 0;
    if (q && p.num_q_heads == 0) return FFD_ERR_INVALID_ARG;
    if (!row_stride(p.k_stride, p.num_kv_heads) || !row_stride(p.v_stride, p.num_kv_heads) ||
        (queries && (!row_stride(p.q_stride, p.num_q_heads) || !row_stride(p.q_out_stride, p.num_q_heads))))
        return FFD_ERR_INVALID_ARG;
    for (const void *x : {q, k_new, v_new, (const void *)q_out, (const void *)k, (const void *)v,
                          (const void *)thumb, (const void *)resid})
        if (!aligned(x, 16)) return FFD_ERR_INVALID_ARG;
    for (const void *x : {(const void *)inv_freq, (const void *)rope_positions, (const void *)cu_tokens,
                          (const void *)positions, (const void *)block_table, (const void *)error_word})
        if (!aligned(x, 4)) return FFD_ERR_INVALID_ARG;
    if (p.head_dim != kD || p.page_size != kPage) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)p.max_blocks_per_seq * kPage > INT32_MAX) return FFD_ERR_UNSUPPORTED;
    if (thumb && p.dtype != FFD_DTYPE_BF16) return FFD_ERR_UNSUPPORTED;
    const int64_t heads = (int64_t)p.num_q_heads + 2 * (int64_t)p.num_kv_heads;
    if (heads > 65536 || T * ((heads + 7) / 8) > (int64_t)INT32_MAX * 4) return FFD_ERR_UNSUPPORTED;
    // A token's rows are read and written by several warps, at their own times.
    if (T > 0) {
        const int64_t B = p.batch, tiles = (int64_t)p.num_pages * p.num_kv_heads;
        const Rows in[] = {{queries ? q : nullptr, T, p.q_stride, p.num_q_heads},
                           {k_new, T, p.k_stride, p.num_kv_heads}, {v_new, T, p.v_stride, p.num_kv_heads}};
        const Rows out = {queries ? q_out : nullptr, T, p.q_out_stride, p.num_q_heads};
        const Bytes reads[] = {{inv_freq, 2 * p.rot_dim}, {rope_positions, 4 * T}, {cu_tokens, 4 * (B + 1)},
                               {positions, 4 * B}, {block_table, 4 * B * p.max_blocks_per_seq}};
        const Bytes writes[] = {{k, tiles * kPage * 2 * kD}, {v, tiles * kPage * 2 * kD},
                                {thumb, tiles * kThumbRec}, {resid, tiles * kResidRec}, {error_word, 4}};
        const bool same = queries && q == q_out && (p.q_stride == p.q_out_stride || T == 1);
        for (const Rows &x : in)
            if (overlap_any(writes, x) || (!(same && &x == in) && overlap(x, out))) return FFD_ERR_INVALID_ARG;
        for (const Bytes &x : reads)
            if (overlap_any(writes, x) || overlap(out, x)) return FFD_ERR_INVALID_ARG;
        if (overlap_any(writes, out) || overlap_each_other(writes)) return FFD_ERR_INVALID_ARG;
    }
    RopeArgs a{};
    a.B = p.batch;
    a.Hq = queries ? p.num_q_heads : 0;
    a.Hkv = p.num_kv_heads;
    a.P = p.num_pages;
    a.max_blocks = p.max_blocks_per_seq;
    a.T = p.total_tokens;
    a.each = cu_tokens ? 0 : p.total_tokens / p.batch;
    a.rot = p.rot_dim;
    a.interleaved = p.interleaved;
    a.scale = p.rot_scale;
    a.q_stride = p.q_stride;
    a.q_out_stride = p.q_out_stride;
    a.k_stride = p.k_stride;
    a.v_stride = p.v_stride;
    a.q = static_cast<const uint16_t *>(q);
    a.k_new = static_cast<const uint16_t *>(k_new);
    a.v_new = static_cast<const uint16_t *>(v_new);
    a.inv_freq = inv_freq;
    a.places = rope_positions;
    a.cu = cu_tokens;
    a.positions = positions;
    a.block_table = block_table;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k = static_cast<uint16_t *>(k);
    a.v = static_cast<uint16_t *>(v);
    a.thumb = thumb;
    a.resid = resid;
    a.err = error_word;
    return cuda_status(launch_rope_append(a, p.dtype, static_cast<cudaStream_t>(stream)));
}

size_t ffd_tree_workspace_size(const ffd_tree_params *params) {
    Plan pl;
    return make_plan(params, &pl) == FFD_OK ? pl.total : 0;
}

ffd_status ffd_tree_attention(const ffd_tree_params *params, const void *q, const void *k,
                              const void *v, const int32_t *seq_lens, const int32_t *cu_q,
                              const int32_t *parents, const int32_t *block_table,
                              const uint8_t *keep_in, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream) {
    if (!q || !k || !v || !seq_lens || !block_table || !out || !workspace) return FFD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(parents, 4) || !aligned(block_table, 4) ||
        !aligned(lse, 4) || !aligned(workspace, kAlign))
        return FFD_ERR_INVALID_ARG;
    Plan pl;
    const ffd_status st = make_plan(params, &pl);
    if (st != FFD_OK) return st;
    const ffd_tree_params &p = *params;
    if (parents && p.max_q_len > kMaxNodes) return FFD_ERR_UNSUPPORTED;
    if (!cu_q && p.total_q != (int64_t)p.batch * p.max_q_len) return FFD_ERR_INVALID_ARG;
    if (workspace_bytes < pl.total) return FFD_ERR_WORKSPACE;
    const int64_t row = (int64_t)p.num_q_heads * kD, stride = p.q_stride ? p.q_stride : row;
    {  // inputs are read, and parts of the result written, by several CTAs, at their own times
        const int64_t B = p.batch, T = p.total_q, cache = (int64_t)p.num_pages * p.num_kv_heads * kPage * 2 * kD;
        const Rows queries = {q, T, stride, p.num_q_heads};
        const Bytes reads[] = {{k, cache}, {v, cache}, {seq_lens, 4 * B}, {cu_q, 4 * (B + 1)}, {parents, 4 * T},
                               {block_table, 4 * B * p.max_blocks_per_seq},
                               {keep_in, B * p.num_kv_heads * p.max_blocks_per_seq}};
        const Bytes writes[] = {{out, 2 * T * row}, {lse, 4 * T * p.num_q_heads}, {workspace, (int64_t)pl.total}};
        if (overlap_any(writes, queries) || overlap_each_other(writes)) return FFD_ERR_INVALID_ARG;
        for (const Bytes &x : reads)
            if (overlap_any(writes, x)) return FFD_ERR_INVALID_ARG;
    }
    AttnArgs a{};
    a.B = p.batch;
    a.Hq = p.num_q_heads;
    a.Hkv = p.num_kv_heads;
    a.G = p.num_q_heads / p.num_kv_heads;
    a.P = p.num_pages;
    a.max_blocks = p.max_blocks_per_seq;
    a.max_q = p.max_q_len;
    a.total_q = p.total_q;
    a.window = p.window;
    a.q_stride = stride;
    a.shares = pl.shares;
    a.groups = pl.groups;
    auto over = [](uint32_t d) { return d < 2 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); };
    a.over_shares = over(a.shares);
    a.over_groups = over(a.groups);
    a.over_heads = over(a.Hkv);
    a.by_mask = keep_in && pl.by_mask;
    a.tile_nodes = kTileRows / a.G;
    a.item_nodes = a.tile_nodes * pl.tiles;
    a.wide_out = aligned(out, 32);
    a.over_g = (uint32_t)(((uint64_t)1 << 32) / a.G + (((uint64_t)1 << 32) % a.G != 0));
    a.factor = fmaxf(p.sm_scale * 1.4426950408889634f, 1.2e-38f);  // never 0: times -inf it has to stay -inf
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.keep_in = keep_in;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q;
    a.block_table = block_table;
    a.parents = parents;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.err = static_cast<int *>(workspace);
    a.wait_ns = p.wait_limit_us > 0 ? (uint64_t)p.wait_limit_us * 1000ull : kWaitTimeoutNs;
    return cuda_status(launch_tree_attention(a, pl, p.dtype, static_cast<cudaStream_t>(stream)));
}

ffd_status ffd_tree_commit(const ffd_cache_desc *cache, int32_t batch, int32_t max_blocks_per_seq,
                           int32_t total_nodes, const int64_t *draft, const int64_t *target,
                           const int32_t *parents, const int32_t *cu_nodes, const int32_t *seq_lens,
                           const int32_t *block_table, void *k, void *v, uint8_t *thumb,
                           uint8_t *resid, int32_t *path, int32_t *accepted, int64_t *next_token,
                           int32_t *new_lens, int32_t *error_word, void *stream) {
    if (!cache || !seq_lens || !block_table || !accepted || !next_token || !new_lens)
        return FFD_ERR_INVALID_ARG;
    if (cache->num_pages < 1 || cache->num_kv_heads < 1 || batch < 1 || max_blocks_per_seq < 1 ||
        total_nodes < 0)
        return FFD_ERR_INVALID_ARG;
    if (total_nodes > 0 && (!draft || !target || !path)) return FFD_ERR_INVALID_ARG;
    if (!cu_nodes && total_nodes % batch != 0) return FFD_ERR_INVALID_ARG;
    if ((thumb == nullptr) != (resid == nullptr)) return FFD_ERR_INVALID_ARG;
    for (const void *x : {(const void *)k, (const void *)v, (const void *)thumb, (const void *)resid})
        if (!aligned(x, 16)) return FFD_ERR_INVALID_ARG;
    for (const void *x : {(const void *)draft, (const void *)target, (const void *)next_token})
        if (!aligned(x, 8)) return FFD_ERR_INVALID_ARG;
    for (const void *x : {(const void *)parents, (const void *)cu_nodes, (const void *)seq_lens,
                          (const void *)block_table, (const void *)path, (const void *)accepted,
                          (const void *)new_lens, (const void *)error_word})
        if (!aligned(x, 4)) return FFD_ERR_INVALID_ARG;
    if (cache->head_dim != kD || cache->page_size != kPage) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks_per_seq * kPage > INT32_MAX) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)batch * cache->num_kv_heads > INT32_MAX) return FFD_ERR_UNSUPPORTED;  // grid.x
    if (!cu_nodes && total_nodes / batch > kMaxNodes) return FFD_ERR_UNSUPPORTED;
    // every KV head's block reads the inputs, at its own time, and the first head's writes the results
    const int64_t B = batch, T = total_nodes, tiles = (int64_t)cache->num_pages * cache->num_kv_heads;
    const Bytes reads[] = {{draft, 8 * T}, {target, 8 * T}, {parents, 4 * T}, {cu_nodes, 4 * (B + 1)},
                           {seq_lens, 4 * B}, {block_table, 4 * B * max_blocks_per_seq}};
    const Bytes writes[] = {{path, 4 * T}, {accepted, 4 * B}, {next_token, 8 * B}, {new_lens, 4 * B},
                            {k, tiles * kPage * 2 * kD}, {v, tiles * kPage * 2 * kD},
                            {thumb, tiles * kThumbRec}, {resid, tiles * kResidRec}, {error_word, 4}};
    for (const Bytes &x : reads)
        if (overlap_any(writes, x)) return FFD_ERR_INVALID_ARG;
    if (overlap_each_other(writes)) return FFD_ERR_INVALID_ARG;
    CommitArgs a{};
    a.B = batch;
    a.Hkv = cache->num_kv_heads;
    a.P = cache->num_pages;
    a.max_blocks = max_blocks_per_seq;
    a.T = total_nodes;
    a.each = cu_nodes ? 0 : total_nodes / batch;
    a.draft = draft;
    a.target = target;
    a.parents = parents;
    a.cu = cu_nodes;
    a.seq_lens = seq_lens;
    a.block_table = block_table;
    a.k = static_cast<uint8_t *>(k);
    a.v = static_cast<uint8_t *>(v);
    a.thumb = thumb;
    a.resid = resid;
    a.path = path;
    a.accepted = accepted;
    a.next_token = next_token;
    a.new_lens = new_lens;
    a.err = error_word;
    return cuda_status(launch_tree_commit(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
