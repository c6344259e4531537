// api_paged.cu -- the extern "C" entry points of the rotary paged appends and
// of the attention over e4m3 pages: argument checks before any CUDA call, then
// the launches (paged_rope.cu, paged_fp8_attention.cu).
#include <cmath>
#include <cstdint>

#include "carat_internal.cuh"

namespace carat {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

carat_status launch_status(cudaError_t e) { return e == cudaSuccess ? CARAT_OK : CARAT_ERR_CUDA; }

bool pages_ok(int num_pages, const int32_t *page_table, int max_pages, int page_rows) {
    return num_pages >= 1 && page_table && max_pages >= 1 && page_rows >= kTcTileKeys &&
           page_rows % kTcTileKeys == 0 &&
           (long long)num_pages * page_rows < (1LL << 31) &&
           (long long)max_pages * page_rows < (1LL << 31);
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

}  // extern "C"
