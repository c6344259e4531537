// paged_fp8_attention.cu -- decode / verify attention over paged e4m3 caches
// with one scale per block of tokens and KV head.
//
// For query row (j, h) of request b at position p = context_length + j, over
// the positions t in [max(0, p - window + 1), p]:
//     s_t = scale * ks[t] * sum_d q_d e4m3(k_td),
//     out_d = sum_t 2^(s_t - m) vs[t] e4m3(v_td) / sum_t 2^(s_t - m)
// with ks, vs the scales of the token's block.  One CTA per row: eight warps
// take every eighth key with a running maximum and sum each, merged at the end.
#include "carat_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace carat {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float *f) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged_fp8_simple_kernel(const PagedFp8Params p) {
    constexpr int E = D / 32;   // elements a lane holds
    const int h = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const size_t row = ((size_t)b * p.k + j) * p.q_heads + h;
    const long long ctx = p.context_lengths[b];
    if (ctx < 0 || ctx + p.k > p.capacity) {
        if (threadIdx.x == 0) set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
        for (int d = threadIdx.x; d < D; d += blockDim.x) p.out[row * D + d] = 0x7fc0;
        return;
    }
    const int c = h / p.group;
    float q[E], o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = __uint_as_float((uint32_t)p.q[row * D + lane * E + i] << 16);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const long long pos = ctx + j;
    const long long first = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    for (long long t = first + warp; t <= pos; t += kWarps) {
        const long long r = paged_row(p.page_table, p.max_pages, p.page_rows, p.num_pages, b, t);
        if (r < 0) {   // a page outside the pool reads as zeros
            if (lane == 0) set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
            const float mn = fmaxf(m, 0.f), a = exp2f(m - mn);
            l = l * a + exp2f(-mn);
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] *= a;
            m = mn;
            continue;
        }
        const size_t at = ((size_t)r * p.kv_heads + c) * D + lane * E;
        const size_t sc = (size_t)(r / p.block_rows) * p.kv_heads + c;
        float s = 0.f, x[4];
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            e4m3x4_to_f32(*reinterpret_cast<const uint32_t *>(p.k_pages + at + i), x);
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fmaf(q[i + e], x[e], s);
        }
#pragma unroll
        for (int z = 16; z > 0; z >>= 1) s += __shfl_xor_sync(0xffffffffu, s, z);
        s *= p.scale_log2 * p.k_scales[sc];
        const float mn = fmaxf(m, s);
        const float a = exp2f(m - mn), w = exp2f(s - mn);
        l = l * a + w;
        const float wv = w * p.v_scales[sc];
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            e4m3x4_to_f32(*reinterpret_cast<const uint32_t *>(p.v_pages + at + i), x);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i + e] = fmaf(wv, x[e], o[i + e] * a);
        }
        m = mn;
    }
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i];
    __syncthreads();
    float M = -INFINITY;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    float L = 0.f;
    for (int w = 0; w < kWarps; ++w) L += s_l[w] * (s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M));
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float acc = 0.f;
        for (int w = 0; w < kWarps; ++w)
            acc += s_o[w][d] * (s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M));
        p.out[row * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(acc / L));
    }
}

}  // namespace

bool paged_fp8_supported(int head_dim) { return head_dim == 256 || head_dim == 512; }

size_t paged_fp8_workspace(int batch, int proposal_count, int q_heads, int kv_heads,
                           int head_dim) {
    return batch > 0 ? 256 : 0;
}

cudaError_t launch_paged_fp8_attention(const PagedFp8Params &p, cudaStream_t stream) {
    const dim3 grid(p.q_heads, p.k, p.batch);
    if (p.head_dim == 256)
        paged_fp8_simple_kernel<256><<<grid, kWarps * 32, 0, stream>>>(p);
    else
        paged_fp8_simple_kernel<512><<<grid, kWarps * 32, 0, stream>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace carat
