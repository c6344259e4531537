// api_paged.cu -- the extern "C" entry points of the rotary paged appends and
// of the attention over e4m3 pages: argument checks before any CUDA call, then
// the launches (paged_rope.cu, paged_fp8_attention.cu).
#include <cmath>
#include <cstdint>

#include "carat_internal.cuh"

namespace carat {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

carat_status launch_status(cudaError_t e) { return e == cudaSuccess ? CARAT_OK : CARAT_ERR_CUDA; }

bool page_sizes_ok(int num_pages, int max_pages, int page_rows) {
    return num_pages >= 1 && max_pages >= 1 && page_rows >= kTcTileKeys &&
           page_rows % kTcTileKeys == 0 &&
           (long long)num_pages * page_rows < (1LL << 31) &&
           (long long)max_pages * page_rows < (1LL << 31);
}

bool pages_ok(int num_pages, const int32_t *page_table, int max_pages, int page_rows) {
    return page_table && page_sizes_ok(num_pages, max_pages, page_rows);
}

bool block_rows_ok(int r) { return r == 16 || r == 32 || r == 64 || r == 128; }

// Checks shared by the two rotary appends.
carat_status check_rope(const RopeParams &p) {
    if (p.batch < 0 || p.k < 1 || p.q_heads < 0 || p.kv_heads < 1 || p.head_dim < 16 ||
        p.head_dim % 16 != 0 || p.rotary_dim < 16 || p.rotary_dim % 16 != 0 ||
        p.rotary_dim > p.head_dim || p.table_rows < 1)
        return CARAT_ERR_INVALID_ARG;
    if (!pages_ok(p.num_pages, p.page_table, p.max_pages, p.page_rows) ||
        (long long)p.k > (long long)p.max_pages * p.page_rows)
        return CARAT_ERR_INVALID_ARG;
    if (p.kv_stride < (long long)p.kv_heads * p.head_dim || p.kv_stride % 8 != 0)
        return CARAT_ERR_INVALID_ARG;
    if (p.q_heads > 0 && (p.q_stride < (long long)p.q_heads * p.head_dim || p.q_stride % 8 != 0))
        return CARAT_ERR_INVALID_ARG;
    if ((long long)p.batch * p.k >= (1LL << 31) || (long long)p.kv_heads * p.head_dim > (1 << 24) ||
        (long long)p.q_heads * p.head_dim > (1 << 24))
        return CARAT_ERR_INVALID_ARG;
    if (!rope_shape_ok(p.head_dim)) return CARAT_ERR_UNSUPPORTED;
    if (p.batch == 0) return CARAT_OK;
    if (!p.k_pages || !p.v_pages || !p.k_new || !p.v_new || !p.table || !p.context_lengths ||
        (p.q_heads > 0 && (!p.q || !p.q_out)))
        return CARAT_ERR_INVALID_ARG;
    if (!aligned16(p.k_pages) || !aligned16(p.v_pages) || !aligned16(p.k_new) ||
        !aligned16(p.v_new) || !aligned16(p.table) ||
        (p.q_heads > 0 && (!aligned16(p.q) || !aligned16(p.q_out))))
        return CARAT_ERR_INVALID_ARG;
    return CARAT_OK;
}

RopeParams rope_params(void *key_pages, void *value_pages, int num_pages,
                       const int32_t *page_table, int max_pages, int page_rows,
                       const void *k_new, const void *v_new, int64_t kv_token_stride,
                       void *queries_out, const void *queries, int64_t q_token_stride,
                       const float *cos_sin, int table_rows, int rotary_dim, int interleaved,
                       const int32_t *positions, const int32_t *new_counts,
                       const int32_t *context_lengths, int proposal_count, int batch, int q_heads,
                       int kv_heads, int head_dim) {
    RopeParams p{};
    p.q = static_cast<const uint16_t *>(queries);
    p.q_out = static_cast<uint16_t *>(queries_out);
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.q_stride = q_token_stride;
    p.kv_stride = kv_token_stride;
    p.k_pages = key_pages;
    p.v_pages = value_pages;
    p.table = cos_sin;
    p.positions = positions;
    p.new_counts = new_counts;
    p.context_lengths = context_lengths;
    p.page_table = page_table;
    p.table_rows = table_rows;
    p.rotary_dim = rotary_dim;
    p.interleaved = interleaved;
    p.batch = batch;
    p.k = proposal_count;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.max_pages = max_pages;
    p.page_rows = page_rows;
    p.num_pages = num_pages;
    return p;
}

}  // namespace
}  // namespace carat

using namespace carat;

extern "C" {

carat_status carat_paged_rope_append(void *key_pages, void *value_pages, int num_pages,
                                     const int32_t *page_table, int max_pages, int page_rows,
                                     const void *k_new, const void *v_new, int64_t kv_token_stride,
                                     void *queries_out, const void *queries, int64_t q_token_stride,
                                     const float *cos_sin, int table_rows, int rotary_dim,
                                     int interleaved, const int32_t *positions,
                                     const int32_t *new_counts, const int32_t *context_lengths,
                                     int proposal_count, int batch, int q_heads, int kv_heads,
                                     int head_dim, void *stream) {
    RopeParams p = rope_params(key_pages, value_pages, num_pages, page_table, max_pages, page_rows,
                               k_new, v_new, kv_token_stride, queries_out, queries, q_token_stride,
                               cos_sin, table_rows, rotary_dim, interleaved, positions, new_counts,
                               context_lengths, proposal_count, batch, q_heads, kv_heads, head_dim);
    const carat_status st = check_rope(p);
    if (st != CARAT_OK || batch == 0) return st;
    p.dev_status = device_status_ptr();
    return launch_status(launch_rope_append(p, static_cast<cudaStream_t>(stream)));
}

carat_status carat_paged_rope_append_fp8(
    void *key_pages, void *value_pages, float *k_scales, float *v_scales, int num_pages,
    const int32_t *page_table, int max_pages, int page_rows, int block_rows, const void *k_new,
    const void *v_new, int64_t kv_token_stride, void *queries_out, const void *queries,
    int64_t q_token_stride, const float *cos_sin, int table_rows, int rotary_dim, int interleaved,
    const int32_t *positions, const int32_t *new_counts, const int32_t *context_lengths,
    int proposal_count, int batch, int q_heads, int kv_heads, int head_dim, void *stream) {
    RopeParams p = rope_params(key_pages, value_pages, num_pages, page_table, max_pages, page_rows,
                               k_new, v_new, kv_token_stride, queries_out, queries, q_token_stride,
                               cos_sin, table_rows, rotary_dim, interleaved, positions, new_counts,
                               context_lengths, proposal_count, batch, q_heads, kv_heads, head_dim);
    if (!block_rows_ok(block_rows)) return CARAT_ERR_INVALID_ARG;
    const carat_status st = check_rope(p);
    if (st != CARAT_OK || batch == 0) return st;
    if (!k_scales || !v_scales) return CARAT_ERR_INVALID_ARG;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_rows = block_rows;
    p.dev_status = device_status_ptr();
    return launch_status(launch_rope_append_fp8(p, static_cast<cudaStream_t>(stream)));
}

// Sizes the attention over e4m3 pages takes (capacity: rows of one request).
static carat_status check_paged_fp8(int batch, int proposal_count, int q_heads, int kv_heads,
                                    int head_dim, long long capacity) {
    if (batch < 0 || proposal_count < 1 || proposal_count > kMaxProposals || q_heads < 1 ||
        kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1 || capacity < proposal_count ||
        capacity >= (1LL << 31))
        return CARAT_ERR_INVALID_ARG;
    const int group = q_heads / kv_heads;
    if (!paged_fp8_supported(head_dim) || group > 64 ||
        (long long)group * proposal_count > kMaxTileRows ||
        (long long)batch * q_heads * proposal_count >= (1LL << 24) ||
        (long long)batch * kv_heads * (capacity / kTcTileKeys + 4) >= (1LL << 29))
        return CARAT_ERR_UNSUPPORTED;
    return CARAT_OK;
}

size_t carat_paged_fp8_workspace_bytes(int batch, int proposal_count, int q_heads, int kv_heads,
                                       int head_dim, int capacity) {
    if (check_paged_fp8(batch, proposal_count, q_heads, kv_heads, head_dim, capacity) != CARAT_OK)
        return 0;
    return paged_fp8_workspace(batch, proposal_count, q_heads, kv_heads, head_dim);
}

carat_status carat_paged_verify_attention_fp8(
    void *out, const void *queries, const void *key_pages, const void *value_pages,
    const float *k_scales, const float *v_scales, int num_pages, const int32_t *page_table,
    int max_pages, int page_rows, int block_rows, const int32_t *new_counts,
    const int32_t *context_lengths, int proposal_count, int batch, int q_heads, int kv_heads,
    int head_dim, int window, float scale, void *workspace, size_t workspace_bytes, void *stream) {
    if (!pages_ok(num_pages, page_table, max_pages, page_rows) || !block_rows_ok(block_rows) ||
        window < 0 || !std::isfinite(scale))
        return CARAT_ERR_INVALID_ARG;
    const long long capacity = (long long)max_pages * page_rows;
    carat_status st =
        check_paged_fp8(batch, proposal_count, q_heads, kv_heads, head_dim, capacity);
    if (st != CARAT_OK || batch == 0) return st;
    if (!out || !queries || !key_pages || !value_pages || !k_scales || !v_scales ||
        !context_lengths)
        return CARAT_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(queries) || !aligned16(key_pages) || !aligned16(value_pages))
        return CARAT_ERR_INVALID_ARG;
    const size_t need =
        paged_fp8_workspace(batch, proposal_count, q_heads, kv_heads, head_dim);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return CARAT_ERR_WORKSPACE;
    PagedFp8Params p{};
    p.out = static_cast<uint16_t *>(out);
    p.q = static_cast<const uint16_t *>(queries);
    p.k_pages = static_cast<const uint8_t *>(key_pages);
    p.v_pages = static_cast<const uint8_t *>(value_pages);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.page_table = page_table;
    p.new_counts = new_counts;
    p.context_lengths = context_lengths;
    p.workspace = workspace;
    p.dev_status = device_status_ptr();
    p.max_pages = max_pages;
    p.page_rows = page_rows;
    p.num_pages = num_pages;
    p.block_rows = block_rows;
    p.batch = batch;
    p.k = proposal_count;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.group = q_heads / kv_heads;
    p.capacity = (int)capacity;
    p.window = window;
    p.scale_log2 = scale * 1.4426950408889634f;
    return launch_status(launch_paged_fp8_attention(p, static_cast<cudaStream_t>(stream)));
}

// Requests are looked through 32 at a time, 0.7 us each, while the kernel's other roles wait 2 s
// at most: 0.1 s for this many without a token (22 ms measured for 2^20), 5.7 s for 2^28.
constexpr int kMostRequests = 1 << 22;

// Sizes the attention of a chunk takes.
static carat_status check_paged_chunk(int batch, int k, int q_heads, int kv_heads, int head_dim) {
    if (batch < 0 || k < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 ||
        head_dim < 1)
        return CARAT_ERR_INVALID_ARG;
    if (!paged_chunk_supported(head_dim) || q_heads / kv_heads > 64 || batch > kMostRequests ||
        (long long)batch * k > (1LL << 28) / q_heads || (long long)kv_heads * head_dim > (1 << 24))
        return CARAT_ERR_UNSUPPORTED;
    return CARAT_OK;
}

size_t carat_paged_chunk_workspace_bytes(int batch, int proposal_count, int q_heads, int kv_heads,
                                         int head_dim) {
    if (check_paged_chunk(batch, proposal_count, q_heads, kv_heads, head_dim) != CARAT_OK ||
        batch == 0)
        return 0;
    return paged_chunk_workspace(batch, proposal_count, q_heads, kv_heads, head_dim);
}

carat_status carat_paged_chunk_attention(
    void *out, const void *queries, const void *key_pages, const void *value_pages, int num_pages,
    const int32_t *page_table, int max_pages, int page_rows, const int32_t *new_counts,
    const int32_t *context_lengths, int proposal_count, int batch, int q_heads, int kv_heads,
    int head_dim, int window, int sinks, float scale, void *workspace, size_t workspace_bytes,
    void *stream) {
    if (!page_sizes_ok(num_pages, max_pages, page_rows) || window < 0 || sinks < 0 ||
        !std::isfinite(scale))
        return CARAT_ERR_INVALID_ARG;
    const long long capacity = (long long)max_pages * page_rows;
    carat_status st = check_paged_chunk(batch, proposal_count, q_heads, kv_heads, head_dim);
    if (st != CARAT_OK) return st;
    if (proposal_count > capacity) return CARAT_ERR_INVALID_ARG;
    if (batch == 0) return CARAT_OK;
    if (!out || !queries || !key_pages || !value_pages || !page_table || !context_lengths)
        return CARAT_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(queries) || !aligned16(key_pages) || !aligned16(value_pages))
        return CARAT_ERR_INVALID_ARG;
    const size_t need = paged_chunk_workspace(batch, proposal_count, q_heads, kv_heads, head_dim);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return CARAT_ERR_WORKSPACE;
    // a pair writes rows while another still reads
    const size_t out_bytes = (size_t)batch * proposal_count * q_heads * head_dim * 2;
    const size_t page_bytes = (size_t)num_pages * page_rows * kv_heads * head_dim * 2;
    if (overlap(out, out_bytes, queries, out_bytes) ||
        overlap(out, out_bytes, key_pages, page_bytes) ||
        overlap(out, out_bytes, value_pages, page_bytes) ||
        (need > 0 && overlap(out, out_bytes, workspace, need)))
        return CARAT_ERR_INVALID_ARG;
    PagedChunkParams p{};
    p.out = static_cast<uint16_t *>(out);
    p.q = static_cast<const uint16_t *>(queries);
    p.k_pages = static_cast<const uint16_t *>(key_pages);
    p.v_pages = static_cast<const uint16_t *>(value_pages);
    p.page_table = page_table;
    p.new_counts = new_counts;
    p.context_lengths = context_lengths;
    p.workspace = workspace;
    p.dev_status = device_status_ptr();
    p.max_pages = max_pages;
    p.page_rows = page_rows;
    p.num_pages = num_pages;
    p.batch = batch;
    p.k = proposal_count;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.group = q_heads / kv_heads;
    p.capacity = (int)capacity;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    return launch_status(launch_paged_chunk_attention(p, static_cast<cudaStream_t>(stream)));
}

constexpr int kMostJobs = 1 << 30;   // a CTA's next job still fits an int

// What the operators on pages share: the pool's geometry and arrays.  Without pages (a
// move whose bytes are moved already) only the scales are looked at.
static carat_status pages_params(PagesParams *p, bool need_pages, void *key_pages,
                                 void *value_pages, float *k_scales, float *v_scales,
                                 int num_pages, int page_rows, int64_t row_bytes, int block_rows,
                                 int kv_heads, int count) {
    if (num_pages < 1 || page_rows < 1 || row_bytes < 16 || row_bytes % 16 != 0 || count < 0 ||
        count > kMostJobs || row_bytes > (1LL << 40) / page_rows)
        return CARAT_ERR_INVALID_ARG;
    if ((k_scales == nullptr) != (v_scales == nullptr) ||
        (k_scales && (block_rows < 1 || page_rows % block_rows != 0 || kv_heads < 1 ||
                      (long long)(page_rows / block_rows) * kv_heads > (1 << 28))))
        return CARAT_ERR_INVALID_ARG;
    if (count == 0) return CARAT_OK;
    if (!key_pages != !value_pages || (need_pages && !key_pages)) return CARAT_ERR_INVALID_ARG;
    if (!aligned16(key_pages) || !aligned16(value_pages)) return CARAT_ERR_INVALID_ARG;
    p->key_pages = key_pages;
    p->value_pages = value_pages;
    p->k_scales = k_scales;
    p->v_scales = v_scales;
    p->num_pages = num_pages;
    p->page_rows = page_rows;
    p->row_bytes = row_bytes;
    p->block_rows = block_rows;
    p->kv_heads = kv_heads;
    p->count = count;
    return CARAT_OK;
}

carat_status carat_pages_copy(void *key_pages, void *value_pages, float *k_scales, float *v_scales,
                              int num_pages, int page_rows, int64_t row_bytes, int block_rows,
                              int kv_heads, const int32_t *src, const int32_t *dst,
                              const int32_t *rows, int count, void *stream) {
    PagesParams p{};
    const carat_status st = pages_params(&p, true, key_pages, value_pages, k_scales, v_scales,
                                         num_pages, page_rows, row_bytes, block_rows, kv_heads,
                                         count);
    if (st != CARAT_OK || count == 0) return st;
    if (!src || !dst) return CARAT_ERR_INVALID_ARG;
    p.src = src;
    p.dst = dst;
    p.rows = rows;
    p.dev_status = device_status_ptr();
    return launch_status(launch_pages_copy(p, static_cast<cudaStream_t>(stream)));
}

carat_status carat_paged_fork(void *key_pages, void *value_pages, float *k_scales, float *v_scales,
                              int num_pages, int page_rows, int64_t row_bytes, int block_rows,
                              int kv_heads, const int32_t *page_table, int num_parents,
                              int max_pages, const int32_t *context_lengths, int32_t *child_table,
                              int32_t *child_lengths, const int32_t *parents,
                              const int32_t *new_pages, int children, void *stream) {
    PagesParams p{};
    const carat_status st = pages_params(&p, true, key_pages, value_pages, k_scales, v_scales,
                                         num_pages, page_rows, row_bytes, block_rows, kv_heads,
                                         children);
    if (st != CARAT_OK) return st;
    if (num_parents < 1 || num_parents > kMostJobs || max_pages < 1 || (long long)max_pages * page_rows >= (1LL << 31))
        return CARAT_ERR_INVALID_ARG;
    if (children == 0) return CARAT_OK;
    if (!page_table || !context_lengths || !child_table || !parents || !new_pages)
        return CARAT_ERR_INVALID_ARG;
    // a child's line written while another child's parent is read from it
    const size_t line = (size_t)max_pages * sizeof(int32_t);
    if (overlap(page_table, num_parents * line, child_table, children * line) ||
        (child_lengths && overlap(context_lengths, (size_t)num_parents * 4, child_lengths,
                                  (size_t)children * 4)))
        return CARAT_ERR_INVALID_ARG;
    p.page_table = page_table;
    p.num_parents = num_parents;
    p.max_pages = max_pages;
    p.context_lengths = context_lengths;
    p.child_table = child_table;
    p.child_lengths = child_lengths;
    p.parents = parents;
    p.new_pages = new_pages;
    p.dev_status = device_status_ptr();
    return launch_status(launch_paged_fork(p, static_cast<cudaStream_t>(stream)));
}

carat_status carat_pages_move(void *key_pages, void *value_pages, float *k_scales, float *v_scales,
                              int num_pages, int page_rows, int64_t row_bytes, int block_rows,
                              int kv_heads, const int32_t *src, const int32_t *dst, int count,
                              int32_t *page_table, int64_t table_entries, void *stream) {
    PagesParams p{};
    const carat_status st = pages_params(&p, false, key_pages, value_pages, k_scales, v_scales,
                                         num_pages, page_rows, row_bytes, block_rows, kv_heads,
                                         count);
    if (st != CARAT_OK) return st;
    if (table_entries < 0 || table_entries >= (1LL << 40) || (table_entries > 0 && !page_table))
        return CARAT_ERR_INVALID_ARG;
    if (count == 0) return CARAT_OK;
    if (!src || !dst) return CARAT_ERR_INVALID_ARG;
    p.src = src;
    p.dst = dst;
    p.table = page_table;
    p.table_entries = table_entries;
    p.dev_status = device_status_ptr();
    return launch_status(launch_pages_move(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
