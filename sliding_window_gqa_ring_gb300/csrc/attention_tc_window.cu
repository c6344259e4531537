// attention_tc_window.cu -- the stream-K attention over bf16 pages under a window with first
// tokens that stay visible (kPagedWindow): the few-row form of the attention of a chunk.
// A request's few rows are the products' short side (16 to 64), its keys the long one: the bound
// is the keys' and values' bytes.  64 requests of 4 tokens under a window of 4096 with 16 first
// tokens take 157 us, 67% of the copy rate (104.7 us); where the pairs of paged_chunk.cu take
// over is at few_rows there.
// Compiled apart from attention_tc.cu so the builds run side by side.
#include "attention_tc.cuh"

namespace carat {

bool tc_window_supported(int head_dim, int group, int k) {
    return head_dim == 512 && group * k <= 64;
}

cudaError_t launch_attention_tc_window(const AttnParams &p, int grid, cudaStream_t stream) {
    TcPlan plan{};
    plan.row_groups = 1;
    plan.pos_per_group = p.k;
    TcMaps maps{};
    const uint64_t D = (uint64_t)p.head_dim;
    const uint64_t dims_kv[4] = {64, (uint64_t)p.num_pages * p.page_rows, D / 64,
                                 (uint64_t)p.kv_heads};
    const uint64_t strides_kv[3] = {(uint64_t)p.kv_heads * D * 2, 128, D * 2};
    const uint32_t box_kv[4] = {64, (uint32_t)kTileKeys, 2, 1};
    const uint64_t dims_q[4] = {D, (uint64_t)p.q_heads, (uint64_t)p.k, (uint64_t)p.batch};
    const uint64_t strides_q[3] = {D * 2, (uint64_t)p.q_heads * D * 2,
                                   (uint64_t)p.k * p.q_heads * D * 2};
    const uint32_t box_q[4] = {64, (uint32_t)p.group, (uint32_t)p.k, 1};
    if (!make_bf16_tensor_map(&maps.k, p.k_base, 4, dims_kv, strides_kv, box_kv, true) ||
        !make_bf16_tensor_map(&maps.v, p.v_base, 4, dims_kv, strides_kv, box_kv, true) ||
        !make_bf16_tensor_map(&maps.q, p.q, 4, dims_q, strides_q, box_q, true))
        return cudaErrorInvalidValue;
    maps.disp = maps.knew = maps.k;
    maps.vnew = maps.v;
    const int n = tc_rows_per_tile(p.group, p.k);
    if (n == 16) return launch_tc<512, 16, 4, 1, 0, false, true>(p, plan, maps, grid, stream);
    if (n == 32) return launch_tc<512, 32, 5, 1, 0, false, true>(p, plan, maps, grid, stream);
    return launch_tc<512, 64, 4, 1, 0, false, true>(p, plan, maps, grid, stream);
}

}  // namespace carat
