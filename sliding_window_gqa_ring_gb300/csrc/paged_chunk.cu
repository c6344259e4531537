// paged_chunk.cu -- attention of a chunk of new tokens over bf16 pages.
//
// Query j of request b sits at position p = context_lengths[b] + j and sees key t when
//   t <= p  and  (window == 0  or  t > p - window  or  t < sinks);
//   out = sum_t softmax_t(scale q . k_t) v_t over the keys it sees.
//
// One warp a query row, one pass over its keys with the running maximum and sum of a
// softmax in fp32: simple, and far from the tensor cores' rate.
#include "carat_internal.cuh"

#include <cmath>

#include <cuda_bf16.h>

namespace carat {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;

struct Request {
    long long ctx;
    int n;
};

__device__ __forceinline__ Request load_request(const PagedChunkParams &p, int b) {
    return {p.context_lengths[b], p.new_counts ? p.new_counts[b] : p.k};
}

__device__ __forceinline__ bool request_ok(const PagedChunkParams &p, const Request &r) {
    return r.ctx >= 0 && r.n >= 0 && r.n <= p.k && r.ctx + r.n <= p.capacity;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) paged_chunk_kernel(const PagedChunkParams p) {
    constexpr int E = D / 32;   // elements of the row a lane holds
    wait_for_prior_launch();
    let_next_launch_start();
    const int lane = threadIdx.x % 32;
    const long long row = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    if (row >= (long long)p.batch * p.k * p.q_heads) return;
    const int h = (int)(row % p.q_heads);
    const int j = (int)(row / p.q_heads % p.k), b = (int)(row / p.q_heads / p.k);
    const Request rq = load_request(p, b);
    uint16_t *out = p.out + row * D + lane * E;
    if (!request_ok(p, rq)) {
        if (lane == 0) set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
        for (int i = 0; i < E; ++i) out[i] = 0x7fff;
        return;
    }
    if (j >= rq.n) return;
    const int c = h / p.group;
    float q[E], o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = __uint_as_float((uint32_t)p.q[row * D + lane * E + i] << 16);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const long long pos = rq.ctx + j;
    const long long first = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    const long long sinks = p.sinks < first ? p.sinks : first;
    for (long long x = 0; x < sinks + pos + 1 - first; ++x) {
        const long long t = x < sinks ? x : first + x - sinks;
        const long long at = paged_row(p.page_table, p.max_pages, p.page_rows, p.num_pages, b, t);
        if (at < 0 && lane == 0) set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
        const size_t off = ((size_t)(at < 0 ? 0 : at) * p.kv_heads + c) * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i)
            s += q[i] * (at < 0 ? 0.f : __uint_as_float((uint32_t)p.k_pages[off + i] << 16));
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(kFull, s, i);
        s *= p.scale_log2;
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - top);
        const float w = exp2f(s - top);
        l = l * keep + w;
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] = o[i] * keep +
                   w * (at < 0 ? 0.f : __uint_as_float((uint32_t)p.v_pages[off + i] << 16));
        m = top;
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        out[i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] / l));
}

}  // namespace

bool paged_chunk_supported(int head_dim) { return head_dim == 256 || head_dim == 512; }

size_t paged_chunk_workspace(int, int, int, int, int) { return 0; }

cudaError_t launch_paged_chunk_attention(const PagedChunkParams &p, cudaStream_t stream) {
    const long long rows = (long long)p.batch * p.k * p.q_heads;
    const dim3 grid((unsigned)((rows + kWarps - 1) / kWarps));
    return launch_dependent(p.head_dim == 256 ? paged_chunk_kernel<256> : paged_chunk_kernel<512>,
                            grid, dim3(32 * kWarps), 0, stream, p);
}

}  // namespace carat
