// paged_rope.cu -- this step's rows into a paged cache, with the rotary
// position embedding applied on the way: into bf16 pages, or into e4m3 pages
// with one scale per block of tokens and KV head.
//
// Rotation.  With c_i, s_i the table's cosine and sine of the token's
// position for frequency i < rotary_dim / 2, a pair (a, b) becomes
// (a c_i - b s_i, b c_i + a s_i); the pair is (x_i, x_{i + rotary_dim/2})
// (half-split) or (x_2i, x_2i+1) (interleaved).  A thread takes 16 elements,
// eight pairs: two 16-byte pieces, half a rotated part apart (half-split) or
// adjacent (interleaved, and the elements past rotary_dim, which pass
// unrotated), so both styles load and store 16 bytes at a time and read the
// same eight cosines and sines.  fp32 throughout, rounded once at the end.
#include "carat_internal.cuh"

#include <cuda_bf16.h>

namespace carat {
namespace {

constexpr int kThreads = 256;
constexpr int kExpMin = -100, kExpMax = 100;   // exponents of the block scales

// One request of the call.
struct Request {
    long long ctx;   // tokens before this step
    int n;           // rows it appends
    bool ok;
};

__device__ __forceinline__ Request load_request(const RopeParams &p, int b) {
    Request r;
    r.ctx = p.context_lengths[b];
    r.n = p.new_counts ? p.new_counts[b] : p.k;
    r.ok = r.ctx >= 0 && r.n >= 0 && r.n <= p.k &&
           r.ctx + r.n <= (long long)p.max_pages * p.page_rows;
    return r;
}

// Row of the rotation table for token j of request b, or -1 outside it.
__device__ __forceinline__ long long table_row(const RopeParams &p, int b, int j, long long ctx) {
    const long long pos = p.positions ? (long long)p.positions[(size_t)b * p.k + j] : ctx + j;
    return pos >= 0 && pos < p.table_rows ? pos : -1;
}

// Where a thread's 16 elements of a row of head_dim lie: two pieces of 8.
struct Piece {
    int a, b;      // first elements of the pieces
    int freq;      // first of the eight frequencies; -1: not rotated
};

__device__ __forceinline__ Piece piece_of(const RopeParams &p, int c, bool rotated) {
    Piece t;
    t.a = 16 * c;
    t.b = t.a + 8;
    t.freq = -1;
    if (rotated && t.a < p.rotary_dim) {
        t.freq = 8 * c;
        if (!p.interleaved) {
            t.a = 8 * c;
            t.b = t.a + p.rotary_dim / 2;
        }
    }
    return t;
}

struct Angles {
    float c[8], s[8];
};

__device__ __forceinline__ void load_angles(const RopeParams &p, long long row, int freq,
                                            Angles &a) {
    const float4 *t = reinterpret_cast<const float4 *>(p.table + (size_t)row * p.rotary_dim + freq);
    const float4 *u = t + p.rotary_dim / 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 c = __ldg(t + i), s = __ldg(u + i);
        a.c[4 * i] = c.x, a.c[4 * i + 1] = c.y, a.c[4 * i + 2] = c.z, a.c[4 * i + 3] = c.w;
        a.s[4 * i] = s.x, a.s[4 * i + 1] = s.y, a.s[4 * i + 2] = s.z, a.s[4 * i + 3] = s.w;
    }
}

__device__ __forceinline__ void widen8(const uint4 &w, float *x) {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
}

// x[0..8) and x[8..16): the thread's pieces, rotated in place.
__device__ __forceinline__ void rotate16(float (&x)[16], const Angles &a, bool interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : i + 8;
        const float u = x[ia], v = x[ib];
        x[ia] = fmaf(u, a.c[i], -(v * a.s[i]));
        x[ib] = fmaf(v, a.c[i], u * a.s[i]);
    }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 narrow8(const float *x) {
    return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]),
                      bf16x2(x[6], x[7]));
}

// One thread's part of token (b, j)'s rows in a bf16 launch: chunks of 16
// elements first, first + step, ... of the row of `heads` heads (queries,
// then with `cache` keys and values).  step is a multiple of head_dim / 16,
// so a thread keeps its place within a head and loads its angles once.
__device__ __forceinline__ void move_token(const RopeParams &p, int b, int j, const Request &rq,
                                           int first, int step, bool cache) {
    const int per = p.head_dim / 16;
    const int c = first % per;
    const size_t token = (size_t)b * p.k + j;
    const bool live = j < rq.n;
    long long trow = -1, drow = -1;
    if (rq.ok && live) {
        trow = table_row(p, b, j, rq.ctx);
        if (cache && trow >= 0)
            drow = paged_row(p.page_table, p.max_pages, p.page_rows, p.num_pages, b, rq.ctx + j);
        if (first == 0) {
            if (trow < 0) set_status(p.dev_status, CARAT_DEV_BAD_POSITION);
            else if (cache && drow < 0) set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
        }
    } else if (rq.ok) {
        return;   // a row behind the request's last: nothing is written
    }
    const bool bad = trow < 0;   // rejected request, or a position outside the table
    const Piece turned = piece_of(p, c, true), plain = piece_of(p, c, false);
    Angles ang;
    if (!bad && turned.freq >= 0) load_angles(p, trow, turned.freq, ang);
    const int heads = p.q_heads + (cache ? 2 * p.kv_heads : 0);
    for (int x = first; x < heads * per; x += step) {
        const int h = x / per;
        const bool is_q = h < p.q_heads;
        const bool is_v = h >= p.q_heads + p.kv_heads;
        const int hk = is_q ? h : is_v ? h - p.q_heads - p.kv_heads : h - p.q_heads;
        uint16_t *dst;
        const uint16_t *src;
        if (is_q) {
            src = p.q + token * p.q_stride + (size_t)h * p.head_dim;
            dst = p.q_out + (token * p.q_heads + h) * p.head_dim;
        } else {
            if (drow < 0) continue;
            src = (is_v ? p.v_new : p.k_new) + token * p.kv_stride + (size_t)hk * p.head_dim;
            dst = reinterpret_cast<uint16_t *>(is_v ? p.v_pages : p.k_pages) +
                  ((size_t)drow * p.kv_heads + hk) * p.head_dim;
        }
        const Piece t = is_v ? plain : turned;
        if (bad) {   // only queries come here
            const uint4 nan = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
            *reinterpret_cast<uint4 *>(dst + t.a) = nan;
            *reinterpret_cast<uint4 *>(dst + t.b) = nan;
            continue;
        }
        uint4 wa = *reinterpret_cast<const uint4 *>(src + t.a);
        uint4 wb = *reinterpret_cast<const uint4 *>(src + t.b);
        if (t.freq >= 0) {
            float v[16];
            widen8(wa, v);
            widen8(wb, v + 8);
            rotate16(v, ang, p.interleaved != 0);
            wa = narrow8(v);
            wb = narrow8(v + 8);
        }
        *reinterpret_cast<uint4 *>(dst + t.a) = wa;
        *reinterpret_cast<uint4 *>(dst + t.b) = wb;
    }
}

// bf16 pages: `splits` CTAs per token (b, j).
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p, int splits) {
    const unsigned token = blockIdx.x / splits, part = blockIdx.x % splits;
    const int b = token / p.k, j = token % p.k;
    const Request rq = load_request(p, b);
    if (!rq.ok && threadIdx.x == 0 && part == 0 && j == 0)
        set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
    move_token(p, b, j, rq, part * blockDim.x + threadIdx.x, splits * blockDim.x, true);
}

// Least e in [kExpMin, kExpMax] with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (u < 0x00800000u) e = kExpMin;   // zero or subnormal
    e = min(max(e, kExpMin), kExpMax);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    // cvt packs its first source into the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Four e4m3 bytes times `ratio`, rounded to e4m3 again.
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float ratio) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    float f[4];
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[0]), "=f"(f[1])
        : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2]), "=f"(f[3])
        : "r"(hi));
    return e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// e4m3 pages: CTAs [0, kv_ctas) take one (request, block of block_rows
// positions, KV head, K or V) each, the others the queries of one token.
// A block's scale is one power of two for its rows of one head: the largest
// finite magnitude of this call's rows fixes the exponent, and a block that
// already held rows of this request keeps its scale unless a larger one is
// needed; then its old bytes are rounded once more, which is exact but for
// values that become subnormal (a power of two moves an e4m3 exponent only).
// One CTA owns the block's rows of its head and their scale, so nothing is
// shared between CTAs.
__global__ void __launch_bounds__(kThreads) rope_append_fp8_kernel(const RopeParams p, int blocks,
                                                                   unsigned kv_ctas, int splits) {
    if (blockIdx.x >= kv_ctas) {
        const unsigned id = blockIdx.x - kv_ctas;
        const unsigned token = id / splits, part = id % splits;
        const int b = token / p.k, j = token % p.k;
        const Request rq = load_request(p, b);
        move_token(p, b, j, rq, part * blockDim.x + threadIdx.x, splits * blockDim.x, false);
        return;
    }
    unsigned id = blockIdx.x;
    const bool is_v = id & 1;
    id >>= 1;
    const int h = id % p.kv_heads;
    id /= p.kv_heads;
    const int nb = id % blocks, b = id / blocks;
    const Request rq = load_request(p, b);
    if (!rq.ok) {
        if (threadIdx.x == 0 && nb == 0 && h == 0 && !is_v)
            set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
        return;
    }
    const int R = p.block_rows;
    const long long t0 = (rq.ctx / R + nb) * R;              // the block's first position
    const long long lo = t0 > rq.ctx ? t0 : rq.ctx;          // this call's rows in it
    const long long hi = t0 + R < rq.ctx + rq.n ? t0 + R : rq.ctx + rq.n;
    if (lo >= hi) return;
    const long long row0 =
        paged_row(p.page_table, p.max_pages, p.page_rows, p.num_pages, b, t0);
    if (row0 < 0) {
        if (threadIdx.x == 0) set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
        return;
    }
    const int per = p.head_dim / 16;
    const int rows = blockDim.x / per;   // rows a pass of the CTA covers
    const int c = threadIdx.x % per, r0 = threadIdx.x / per;
    const Piece t = piece_of(p, c, !is_v);
    const uint16_t *src = is_v ? p.v_new : p.k_new;
    uint8_t *dst = reinterpret_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages);
    float *scale_at = (is_v ? p.v_scales : p.k_scales) + (size_t)(row0 / R) * p.kv_heads + h;

    // This thread's 16 values of position pos (false: outside the table).
    auto values = [&](long long pos, float (&x)[16]) -> bool {
        const int j = (int)(pos - rq.ctx);
        const long long trow = table_row(p, b, j, rq.ctx);
        if (trow < 0) return false;
        const uint16_t *s = src + ((size_t)b * p.k + j) * p.kv_stride + (size_t)h * p.head_dim;
        widen8(*reinterpret_cast<const uint4 *>(s + t.a), x);
        widen8(*reinterpret_cast<const uint4 *>(s + t.b), x + 8);
        if (t.freq >= 0) {
            Angles a;
            load_angles(p, trow, t.freq, a);
            rotate16(x, a, p.interleaved != 0);
        }
        return true;
    };

    float amax = 0.f;
    bool any = false, outside = false;
    for (long long pos = lo + r0; pos < hi; pos += rows) {
        float x[16];
        if (!values(pos, x)) {
            outside = true;
            continue;
        }
        any = true;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[i]));
    }
    if (outside && c == 0) set_status(p.dev_status, CARAT_DEV_BAD_POSITION);
    __shared__ float s_max[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = amax;
    if (!__syncthreads_or(any)) return;   // no row of the block is written
    for (int w = 0; w < (int)(blockDim.x + 31) / 32; ++w) amax = fmaxf(amax, s_max[w]);
    const float need = scale_for(amax);
    const bool fresh = t0 >= rq.ctx;
    const float old = fresh ? need : *scale_at;
    const float scale = fmaxf(old, need);
    const float inv = 1.f / scale;
    __syncthreads();   // the old scale is read before it is replaced
    if (threadIdx.x == 0) *scale_at = scale;
    if (scale != old) {
        const float ratio = old * inv;
        for (long long pos = t0 + r0; pos < rq.ctx; pos += rows) {
            uint4 *w = reinterpret_cast<uint4 *>(
                dst + ((size_t)(row0 + (pos - t0)) * p.kv_heads + h) * p.head_dim + 16 * c);
            const uint4 v = *w;
            *w = make_uint4(requantise4(v.x, ratio), requantise4(v.y, ratio),
                            requantise4(v.z, ratio), requantise4(v.w, ratio));
        }
    }
    for (long long pos = lo + r0; pos < hi; pos += rows) {
        float x[16];
        if (!values(pos, x)) continue;
        uint8_t *d = dst + ((size_t)(row0 + (pos - t0)) * p.kv_heads + h) * p.head_dim;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = e4m3x4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv,
                          x[4 * i + 3] * inv);
        *reinterpret_cast<uint2 *>(d + t.a) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2 *>(d + t.b) = make_uint2(o[2], o[3]);
    }
}

// Threads of a CTA: a multiple of the 16-element chunks of a head, so that a
// thread keeps its place within the head, and whole warps.
int cta_threads(int head_dim) {
    const int per = head_dim / 16;
    if (per >= 32 || 32 % per) {
        int t = per;
        while (t % 32) t += per;
        while (t + t <= kThreads) t += t;
        return t;
    }
    return kThreads;
}

// CTAs a token's rows are spread over: enough that a call of few tokens
// gives each thread one chunk.
int token_splits(const RopeParams &p, int heads, int threads) {
    const long long chunks = (long long)heads * (p.head_dim / 16);
    const long long full = (chunks + threads - 1) / threads;
    const long long tokens = (long long)p.batch * p.k;
    const long long want = (8ll * 152 + tokens - 1) / tokens;
    return (int)(want < full ? (want < 1 ? 1 : want) : full);
}

}  // namespace

bool rope_shape_ok(int head_dim) { return head_dim <= 1024 && cta_threads(head_dim) <= kThreads; }

cudaError_t launch_rope_append(const RopeParams &p, cudaStream_t stream) {
    const int threads = cta_threads(p.head_dim);
    const int splits = token_splits(p, p.q_heads + 2 * p.kv_heads, threads);
    const long long grid = (long long)p.batch * p.k * splits;
    if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
    rope_append_kernel<<<(unsigned)grid, threads, 0, stream>>>(p, splits);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_rope_append_fp8(const RopeParams &p, cudaStream_t stream) {
    const int threads = cta_threads(p.head_dim);
    const int splits = p.q_heads > 0 ? token_splits(p, p.q_heads, threads) : 0;
    const int blocks = (p.k + p.block_rows - 2) / p.block_rows + 1;
    const long long kv = (long long)p.batch * blocks * p.kv_heads * 2;
    const long long grid = kv + (long long)p.batch * p.k * splits;
    if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
    rope_append_fp8_kernel<<<(unsigned)grid, threads, 0, stream>>>(p, blocks, (unsigned)kv,
                                                                   splits);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace carat
