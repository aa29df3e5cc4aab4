// kv4_api.cu -- the 4-bit cache's C entries (declared in include/ffd.h): argument checks, workspace
// planning and launches.
#include <math.h>

#include "kv4.cuh"
#include "ptx.cuh"

namespace ffd {
namespace kv4 {
cudaError_t launch_write(const RowsArgs &a, int dtype, const void *k, const void *v, uint8_t *k4,
                         uint8_t *v4, cudaStream_t stream);
cudaError_t launch_read(const RowsArgs &a, int dtype, const uint8_t *k4, const uint8_t *v4, void *k,
                        void *v, cudaStream_t stream);
cudaError_t launch_decode(const AttnArgs &a, const Plan &pl, int dtype, cudaStream_t stream);
cudaError_t launch_chunk(const AttnArgs &a, const Plan &pl, int dtype, cudaStream_t stream);
size_t decode_record_bytes(int cols);
size_t chunk_record_bytes();
int decode_slots();
int chunk_slots();
int chunk_once();
int chunk_rows();
int decode_warps(int cols);
}  // namespace kv4
}  // namespace ffd

using namespace ffd;
using namespace ffd::kv4;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = 1 << 28;  // query tokens of a sequence x G
constexpr size_t kMaxUnits = 65535;  // (sequence, KV head) pairs of an attention call, as ffd.h states

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The checks that a write and a read share.
ffd_status check_rows(const ffd_cache_desc *cache, int32_t dtype, int32_t batch, int32_t max_blocks,
                      int32_t total, const void *k, int64_t k_stride, const void *v,
                      int64_t v_stride, const int32_t *cu, const int32_t *positions,
                      const int32_t *block_table, const uint8_t *k4, const uint8_t *v4,
                      const int32_t *error_word) {
    if (!cache || !positions || !block_table) return FFD_ERR_INVALID_ARG;
    if (cache->num_pages < 1 || cache->num_kv_heads < 1 || batch < 1 || max_blocks < 1 || total < 0)
        return FFD_ERR_INVALID_ARG;
    if (cache->head_dim != kD || cache->page_size != kPage) return FFD_ERR_UNSUPPORTED;
    if (dtype != FFD_DTYPE_BF16 && dtype != FFD_DTYPE_F16) return FFD_ERR_INVALID_ARG;
    if (!cu && total % batch != 0) return FFD_ERR_INVALID_ARG;
    const int64_t row = (int64_t)cache->num_kv_heads * kD;
    if (k && (k_stride < row || k_stride % 8 != 0 || !k4)) return FFD_ERR_INVALID_ARG;
    if (v && (v_stride < row || v_stride % 8 != 0 || !v4)) return FFD_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k4, 16) || !aligned(v4, 16) ||
        !aligned(cu, 4) || !aligned(positions, 4) || !aligned(block_table, 4) || !aligned(error_word, 4))
        return FFD_ERR_INVALID_ARG;
    if ((int64_t)max_blocks * kPage > INT32_MAX) return FFD_ERR_UNSUPPORTED;
    if (cache->num_kv_heads > 65535) return FFD_ERR_UNSUPPORTED;  // grid.y
    return FFD_OK;
}

RowsArgs rows_args(const ffd_cache_desc *cache, int32_t batch, int32_t max_blocks, int32_t total,
                   int64_t k_stride, int64_t v_stride, const int32_t *cu, const int32_t *positions,
                   const int32_t *block_table, int32_t *error_word) {
    RowsArgs a{};
    a.B = batch;
    a.Hkv = cache->num_kv_heads;
    a.P = cache->num_pages;
    a.max_blocks = max_blocks;
    a.T = total;
    a.per = cu ? 0 : total / batch;
    a.cu = cu;
    a.positions = positions;
    a.block_table = block_table;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.err = error_word;
    return a;
}

ffd_status check_params(const ffd_kv4_params *p) {
    if (!p) return FFD_ERR_INVALID_ARG;
    if (p->batch < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_pages < 1 ||
        p->max_blocks_per_seq < 1 || p->max_q_len < 1 || p->total_q < 1 || p->window < 0 ||
        p->num_splits < 0 || p->wait_limit_us < 0)
        return FFD_ERR_INVALID_ARG;
    if (p->dtype != FFD_DTYPE_BF16 && p->dtype != FFD_DTYPE_F16) return FFD_ERR_INVALID_ARG;
    if (p->num_q_heads % p->num_kv_heads != 0) return FFD_ERR_INVALID_ARG;
    if (!isfinite(p->sm_scale) || !(p->sm_scale > 0.0f)) return FFD_ERR_INVALID_ARG;
    if (p->q_stride != 0 && (p->q_stride < (int64_t)p->num_q_heads * kD || p->q_stride % 8 != 0))
        return FFD_ERR_INVALID_ARG;
    if (p->head_dim != kD || p->page_size != kPage) return FFD_ERR_UNSUPPORTED;
    if (p->num_q_heads / p->num_kv_heads > kMaxG) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)p->batch * p->num_kv_heads > (int64_t)kMaxUnits) return FFD_ERR_UNSUPPORTED;
    if ((int64_t)p->max_blocks_per_seq * kPage > INT32_MAX) return FFD_ERR_UNSUPPORTED;
    // a record is named by an int32, and so is a page of a unit for each group of rows that takes it
    if ((int64_t)p->num_pages * p->num_kv_heads > INT32_MAX) return FFD_ERR_UNSUPPORTED;
    const int64_t pages = (int64_t)p->batch * p->num_kv_heads * ((int64_t)p->max_blocks_per_seq + kChunkLead);
    const int64_t rows = (int64_t)p->max_q_len * (p->num_q_heads / p->num_kv_heads);
    if (rows > kMaxRows || pages > INT32_MAX ||
        pages > INT32_MAX / ((rows + chunk_rows() - 1) / chunk_rows()))
        return FFD_ERR_UNSUPPORTED;
    return FFD_OK;
}

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// At least this many pages (upper bound from the table's width) for each CTA. Below that what is read side
// by side is lost again in joins: one token over 4096, 2 heads, takes 22, 18, 16, 16, 18, 18 us with 32, 16, 8,
// 4, 2, 1 pages a CTA; nine tokens over 2048, 8 heads, in the chunk kernel 43, 39, 31, 27, 27, 29 with 32, 16,
// 8, 4, 2 and fewer.
constexpr int64_t kMinDecodePages = 8, kMinChunkPages = 4;

// Pages of a cut item that a CTA of the chunk kernel takes at least, for items of n pages: cut in k
// they take n / k pages' time and then that of the records that are joined one after another, k of
// them or, cut in more than chunk_once(), about 2 sqrt(k) in two steps. A record of 256 rows is
// written and joined in about 1.8 pages' time (2200 cycles a page, 4000 a record measured).
int64_t chunk_pages(int64_t n, int64_t rows) {
    const double record = 1.8 * (double)rows / chunk_rows() + 0.2;
    double best = INFINITY;
    int64_t pages = n;
    for (int64_t k = 1; k <= 128 && k * kMinChunkPages <= n; k += k < 8 ? 1 : k / 4) {
        const double joins = k == 1 ? 0.0 : k <= chunk_once() ? k : 2.0 * sqrt((double)k) + 2.0;
        const double time = (double)n / k + record * joins;
        if (time < best) {
            best = time;
            pages = (n + k - 1) / k;
        }
    }
    return pages;
}

// Where whole items (256 rows over the pages they see) are dealt out, `rounds` consecutive ones to a CTA:
// the pages' time that the longest-working CTA has beyond an equal share if all sequences fill the block
// table (the kernel looks at how unequal they are, and cuts the items all the same if they are too much). Some CTAs have an item
// fewer, and the groups of rows of a unit see from first to last as many more pages as there are query
// tokens (less behind a window). While that is less than what cutting costs, whole items are the
// faster way. Measured, us whole and cut, 8 heads and 4 query heads for each:
//   9 sequences of 1024 tokens, their last 128     2 beyond           32   53
//   2 of 4096, 512                                17                  81   84
//   1 of 4096, 1024                               23                  82   88
//   3 of 4096, 256                                28                  82   74
//   8 of 2048, 512                                38, several items   138  149
//   3 of 1024, 1024                               41, several         83   72
//   1 of 8192, 8192                               over 600, several   1024 575
double longest_beyond(const ffd_kv4_params *p, int64_t rounds, int64_t groups, int64_t items, int sms) {
    const int64_t tokens = (int64_t)p->max_blocks_per_seq * kPage;
    const int64_t seen = p->window > 0 && p->window < tokens ? p->window : tokens;
    const int64_t before = tokens > p->max_q_len ? tokens - p->max_q_len : 0;
    const double rise = (double)(seen - (seen < before ? seen : before)) / kPage;
    const double fewer = (double)(rounds * sms - items) * ((double)seen / kPage + kChunkLead) / sms;
    return fewer + (rounds < groups ? 0.75 * rounds * rise * (1.0 - (double)rounds / groups) : 0.0);
}

// Workspace: [error word | three join tickets per CTA | records per CTA | a parked state per warp of
// the decode kernel]. The tickets, the only part that has to start at zero, have the same place and size
// whatever the parameters and are left at zero, so that calls of different shapes can share a
// workspace.
ffd_status make_plan(const ffd_kv4_params *p, Plan *pl) {
    const ffd_status st = check_params(p);
    if (st != FFD_OK) return st;
    const int64_t rows = (int64_t)p->max_q_len * (p->num_q_heads / p->num_kv_heads);
    // Up to 32 rows a KV head the kernel whose warps walk pages alone is the faster one, above it only the
    // one that forms tiles for tcgen05 is left: eight sequences of 5000 to 16384 tokens, 8 heads, take
    // 36, 49, 58 and 86 us for 8, 16, 24 and 32 rows in the first and 90 to 91 us in the second (92 for 36).
    pl->cols = rows <= 32 ? (int)(rows + 7) / 8 * 8 : 0;
    const int sms = current_sm_count();
    const int64_t units = (int64_t)p->batch * p->num_kv_heads;
    const int64_t groups = (rows + chunk_rows() - 1) / chunk_rows(), items = units * groups;
    int64_t ctas = p->num_splits;
    pl->whole_items = 0;
    if (ctas == 0) {
        if (sms <= 0) return FFD_ERR_CUDA;
        if (pl->cols) {
            ctas = (units * p->max_blocks_per_seq + kMinDecodePages - 1) / kMinDecodePages;
        } else {
            const int64_t blocks = p->max_blocks_per_seq;
            const int64_t rounds = (items + sms - 1) / sms;
            int64_t most = blocks;  // pages that an item sees at most
            if (p->window > 0) {
                const int64_t seen = ((int64_t)p->window + p->max_q_len) / kPage + 2;
                most = most < seen ? most : seen;
            }
            if (longest_beyond(p, rounds, groups, items, sms) <=
                (rounds > 1 ? kJoinPagesSeveral : kJoinPages)) {
                pl->whole_items = 1;
                ctas = items;
            } else {
                const int64_t least = chunk_pages(most, rows < chunk_rows() ? rows : chunk_rows());
                ctas = (items * most + least - 1) / least;
            }
        }
    }
    if (sms > 0 && ctas > sms) ctas = sms;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    pl->ctas = (int)ctas;
    // Where work is cut, what an item costs besides its pages counts as well, so that a prompt's many short
    // first items do not come together in a few CTAs (8192 tokens, 32/8 heads: 752 us without, 574 with;
    // 256 rows a head of eight sequences of 5000 to 16384: 122 and 117). Every CTA that begins within an item has such a
    // cost too; with few long items that is nearly all of them, and only those that begin with an item
    // would get fewer pages (256 rows a head of one sequence of 32768: 67.2 us without, 68.6 with).
    pl->lead = pl->cols || 8 * items <= ctas ? 0 : kChunkLead;
    const size_t rec = pl->cols ? decode_record_bytes(pl->cols) : chunk_record_bytes();
    size_t off = kAlign;
    pl->tickets = off;
    off = align_up(off + 3 * kMaxCtas * sizeof(int));
    pl->records = off;
    off = align_up(off + (size_t)(pl->cols ? decode_slots() : chunk_slots()) * pl->ctas * rec);
    pl->parked = off;
    if (pl->cols) off = align_up(off + (size_t)pl->ctas * decode_warps(pl->cols) * rec);
    pl->total = off;
    return FFD_OK;
}

}  // namespace

extern "C" {

ffd_status ffd_kv4_write(const ffd_cache_desc *cache, int32_t dtype, int32_t batch,
                         int32_t max_blocks_per_seq, int32_t total_tokens, const void *k_new,
                         int64_t k_stride, const void *v_new, int64_t v_stride,
                         const int32_t *cu_tokens, const int32_t *positions,
                         const int32_t *block_table, uint8_t *k4, uint8_t *v4,
                         int32_t *error_word, void *stream) {
    if ((!k_new || !v_new) && total_tokens != 0) return FFD_ERR_INVALID_ARG;
    const ffd_status st =
        check_rows(cache, dtype, batch, max_blocks_per_seq, total_tokens, k_new, k_stride, v_new,
                   v_stride, cu_tokens, positions, block_table, k4, v4, error_word);
    if (st != FFD_OK) return st;
    const RowsArgs a = rows_args(cache, batch, max_blocks_per_seq, total_tokens, k_stride, v_stride,
                                 cu_tokens, positions, block_table, error_word);
    return cuda_status(
        launch_write(a, dtype, k_new, v_new, k4, v4, static_cast<cudaStream_t>(stream)));
}

ffd_status ffd_kv4_read(const ffd_cache_desc *cache, int32_t dtype, int32_t batch,
                        int32_t max_blocks_per_seq, int32_t total_tokens, const int32_t *cu_tokens,
                        const int32_t *positions, const int32_t *block_table, const uint8_t *k4,
                        const uint8_t *v4, void *k_out, int64_t k_stride, void *v_out,
                        int64_t v_stride, int32_t *error_word, void *stream) {
    if (!k_out && !v_out && total_tokens != 0) return FFD_ERR_INVALID_ARG;
    const ffd_status st =
        check_rows(cache, dtype, batch, max_blocks_per_seq, total_tokens, k_out, k_stride, v_out,
                   v_stride, cu_tokens, positions, block_table, k4, v4, error_word);
    if (st != FFD_OK) return st;
    const RowsArgs a = rows_args(cache, batch, max_blocks_per_seq, total_tokens, k_stride, v_stride,
                                 cu_tokens, positions, block_table, error_word);
    return cuda_status(
        launch_read(a, dtype, k4, v4, k_out, v_out, static_cast<cudaStream_t>(stream)));
}

size_t ffd_kv4_workspace_size(const ffd_kv4_params *params) {
    Plan pl;
    return make_plan(params, &pl) == FFD_OK ? pl.total : 0;
}

ffd_status ffd_kv4_attention(const ffd_kv4_params *params, const void *q, const uint8_t *k4,
                             const uint8_t *v4, const int32_t *seq_lens, const int32_t *cu_q,
                             const int32_t *block_table, const uint8_t *keep_in, void *out,
                             float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k4 || !v4 || !seq_lens || !block_table || !out || !workspace)
        return FFD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k4, 16) || !aligned(v4, 16) || !aligned(out, 16) ||
        !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(block_table, 4) || !aligned(lse, 4) ||
        !aligned(workspace, kAlign))
        return FFD_ERR_INVALID_ARG;
    Plan pl;
    const ffd_status st = make_plan(params, &pl);
    if (st != FFD_OK) return st;
    const ffd_kv4_params &p = *params;
    if (!cu_q && p.total_q != (int64_t)p.batch * p.max_q_len) return FFD_ERR_INVALID_ARG;
    if (workspace_bytes < pl.total) return FFD_ERR_WORKSPACE;
    const int64_t row = (int64_t)p.num_q_heads * kD, stride = p.q_stride ? p.q_stride : row;
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
    if (q0 < o0 + (uintptr_t)(2 * (int64_t)p.total_q * row) &&
        o0 < q0 + (uintptr_t)(2 * ((p.total_q - 1) * stride + row)))
        return FFD_ERR_INVALID_ARG;  // q is read by several CTAs, at their own times
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
    a.whole_items = pl.whole_items;
    a.lead = pl.lead;
    a.over_g = (uint32_t)(((uint64_t)1 << 32) / a.G + (((uint64_t)1 << 32) % a.G != 0));
    a.q_stride = stride;
    a.sm_scale = p.sm_scale;
    a.q = q;
    a.k4 = k4;
    a.v4 = v4;
    a.keep_in = keep_in;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q;
    a.block_table = block_table;
    a.out = out;
    a.lse = lse;
    a.err = static_cast<int *>(workspace);
    a.wait_ns = p.wait_limit_us > 0 ? (uint64_t)p.wait_limit_us * 1000ull : kWaitTimeoutNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(pl.cols ? launch_decode(a, pl, p.dtype, s)
                               : launch_chunk(a, pl, p.dtype, s));
}

}  // extern "C"
