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

template <bool kInter>
__device__ __forceinline__ Piece piece_of(const RopeParams &p, int c, bool rotated) {
    Piece t;
    t.a = 16 * c;
    t.b = t.a + 8;
    t.freq = -1;
    if (rotated && t.a < p.rotary_dim) {
        t.freq = 8 * c;
        if (!kInter) {
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
template <bool kInter>
__device__ __forceinline__ void rotate16(float (&x)[16], const Angles &a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = kInter ? 2 * i : i, ib = kInter ? 2 * i + 1 : i + 8;
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

// Chunks a thread has in flight in a call of many tokens (one in a call of few,
// see spread), the CTAs of an SM the registers are fitted to, and the rows of an
// e4m3 block in flight.  Measured on 8 ragged prompts of 2048 tokens, 16 + 2 x 8
// heads x 256 (bf16 / e4m3 pages) and a chunk of 8191 tokens, 16 + 2 x 2 heads x
// 512 (e4m3): 3 chunks at 4 CTAs 58.5 / 65.5 / 65.2 us (the bytes at the copy rate: 51.1 /
// 44.8 / 49.4); 4 at 3 CTAs 60.7 / 68.8 / 60.7; 2 at 4 71.0 / 69.9 / 64.4; one at
// a time 81.4 / 95.4 / 71.2.  (With the e4m3 blocks' unturned values compared as bits:
// 58.4 / 63.6 / 62.6.)  Few tokens: 2.7 us for one, 4.8 for 256.
// The interleaved instances fit their 64 registers; the half-split e4m3 ones spill 9 of
// them (36 bytes stored, 64 loaded), the half-split bf16 one of many tokens 1.
constexpr int kFlight = 3, kMany = 4, kFew = 4;
constexpr int kRows = 2;

// One thread's part of token (b, j)'s rows: chunks of 16 elements first,
// first + step, ... of its rows (queries, then with `cache` keys and
// values).  step is a multiple of head_dim / 16, so a thread keeps its place
// within a head and loads its angles once.  The loads of F chunks go out
// before the first is used.
template <bool kInter, int F>
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
    const Piece turned = piece_of<kInter>(p, c, true), plain = piece_of<kInter>(p, c, false);
    const int heads = p.q_heads + (cache ? 2 * p.kv_heads : 0);
    const int hstep = step / per;
    const uint16_t *q = p.q + token * p.q_stride;
    uint16_t *q_out = p.q_out + token * p.q_heads * p.head_dim;
    if (trow < 0) {   // rejected request, or a position outside the table
        const uint4 nan = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        for (int h = first / per; h < p.q_heads; h += hstep) {
            *reinterpret_cast<uint4 *>(q_out + (size_t)h * p.head_dim + turned.a) = nan;
            *reinterpret_cast<uint4 *>(q_out + (size_t)h * p.head_dim + turned.b) = nan;
        }
        return;
    }
    Angles ang;
    if (turned.freq >= 0) load_angles(p, trow, turned.freq, ang);
    // queries, keys and values are one run of heads; where head h comes from
    // and goes to is formed again for the store rather than held in registers
    const int v0 = p.q_heads + p.kv_heads;
    const size_t kv = token * p.kv_stride, at = (size_t)drow * p.kv_heads * p.head_dim;
    const int end = drow < 0 ? p.q_heads : heads;
    for (int h0 = first / per; h0 < end; h0 += F * hstep) {
        uint4 wa[F], wb[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int h = h0 + i * hstep;
            if (h >= end) break;
            const uint16_t *src = h < p.q_heads ? q + h * p.head_dim
                                  : h < v0      ? p.k_new + kv + (h - p.q_heads) * p.head_dim
                                                : p.v_new + kv + (h - v0) * p.head_dim;
            wa[i] = __ldcs(reinterpret_cast<const uint4 *>(src + (h < v0 ? turned.a : plain.a)));
            wb[i] = __ldcs(reinterpret_cast<const uint4 *>(src + (h < v0 ? turned.b : plain.b)));
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int h = h0 + i * hstep;
            if (h >= end) break;
            if (turned.freq >= 0 && h < v0) {
                float v[16];
                widen8(wa[i], v);
                widen8(wb[i], v + 8);
                rotate16<kInter>(v, ang);
                wa[i] = narrow8(v);
                wb[i] = narrow8(v + 8);
            }
            uint16_t *dst =
                h < p.q_heads ? q_out + h * p.head_dim
                : h < v0 ? reinterpret_cast<uint16_t *>(p.k_pages) + at + (h - p.q_heads) * p.head_dim
                         : reinterpret_cast<uint16_t *>(p.v_pages) + at + (h - v0) * p.head_dim;
            *reinterpret_cast<uint4 *>(dst + (h < v0 ? turned.a : plain.a)) = wa[i];
            *reinterpret_cast<uint4 *>(dst + (h < v0 ? turned.b : plain.b)) = wb[i];
        }
    }
}

// How a launch spreads tokens over CTAs: `per_cta` tokens each, or (per_cta 1)
// one token over `splits` CTAs.
struct Spread {
    int per_cta, splits;
    bool many;
};

template <bool kInter, int F>
__device__ __forceinline__ void move_tokens(const RopeParams &p, unsigned cta, Spread s,
                                            bool cache) {
    const int team = blockDim.x / s.per_cta;
    const unsigned token = cta / s.splits * s.per_cta + threadIdx.x / team;
    if (token >= (unsigned)p.batch * p.k) return;
    const int b = token / p.k, j = token % p.k;
    const Request rq = load_request(p, b);
    const int first = cta % s.splits * blockDim.x + threadIdx.x % team;
    if (!rq.ok && first == 0 && j == 0) set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
    move_token<kInter, F>(p, b, j, rq, first, s.splits * team, cache);
}

// bf16 pages.
template <bool kInter, int F>
__global__ void __launch_bounds__(kThreads, F == 1 ? kFew : kMany) rope_append_kernel(
    const __grid_constant__ RopeParams p, Spread s) {
    wait_for_prior_launch();
    let_next_launch_start();
    move_tokens<kInter, F>(p, blockIdx.x, s, true);
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
// shared between CTAs.  The rows are read twice, the second time from cache: kept in
// shared memory in between (cp.async) they cost 75.5 us against 63.5 at 8 x 2048.
template <bool kInter, int F>
__global__ void __launch_bounds__(kThreads, F == 1 ? kFew : kMany) rope_append_fp8_kernel(
    const __grid_constant__ RopeParams p, int blocks, unsigned kv_ctas, Spread s) {
    wait_for_prior_launch();
    let_next_launch_start();
    if (blockIdx.x >= kv_ctas) {
        move_tokens<kInter, F>(p, blockIdx.x - kv_ctas, s, false);
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
    const Piece t = piece_of<kInter>(p, c, !is_v);
    const uint16_t *src = is_v ? p.v_new : p.k_new;
    uint8_t *dst = reinterpret_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages);
    float *scale_at = (is_v ? p.v_scales : p.k_scales) + (size_t)(row0 / R) * p.kv_heads + h;

    // Rows pos, pos + rows, ... (kRows of them) of this thread: loaded together,
    // and their values one by one (false: no such row, or no angle for it).
    uint4 wa[kRows], wb[kRows];
    auto load = [&](long long pos) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (pos + i * rows >= hi) break;
            const uint16_t *s = src + ((size_t)b * p.k + (pos + i * rows - rq.ctx)) * p.kv_stride +
                                (size_t)h * p.head_dim;
            wa[i] = *reinterpret_cast<const uint4 *>(s + t.a);
            wb[i] = *reinterpret_cast<const uint4 *>(s + t.b);
        }
    };
    auto values = [&](int i, long long pos, float (&x)[16]) -> bool {
        if (pos >= hi) return false;
        const long long trow = table_row(p, b, (int)(pos - rq.ctx), rq.ctx);
        if (trow < 0) return false;
        widen8(wa[i], x);
        widen8(wb[i], x + 8);
        if (t.freq >= 0) {
            Angles a;
            load_angles(p, trow, t.freq, a);
            rotate16<kInter>(x, a);
        }
        return true;
    };

    // Largest magnitude of the thread's rows; +inf when one of them may not be
    // finite.  Values that are not turned are compared as bits, two at a time.
    float amax = 0.f;
    uint32_t bits = 0;
    bool any = false, outside = false;
    for (long long pos = lo + r0; pos < hi; pos += kRows * rows) {
        load(pos);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (pos + i * rows >= hi) continue;
            if (table_row(p, b, (int)(pos + i * rows - rq.ctx), rq.ctx) < 0) {
                outside = true;
                continue;
            }
            any = true;
            if (t.freq < 0) {
                const uint32_t w[8] = {wa[i].x, wa[i].y, wa[i].z, wa[i].w,
                                       wb[i].x, wb[i].y, wb[i].z, wb[i].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) bits = __vmaxu2(bits, w[e] & 0x7fff7fffu);
            } else {
                float x[16];
                values(i, pos + i * rows, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
            }
        }
    }
    bits = max(bits & 0xffffu, bits >> 16);
    amax = bits >= 0x7f80u ? INFINITY : fmaxf(amax, __uint_as_float(bits << 16));
    if (outside && c == 0) set_status(p.dev_status, CARAT_DEV_BAD_POSITION);
    __shared__ float s_max[kThreads / 32];
    auto block_max = [&](float v) -> float {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = v;
        __syncthreads();
        for (int w = 0; w < (int)(blockDim.x + 31) / 32; ++w) v = fmaxf(v, s_max[w]);
        return v;
    };
    if (!__syncthreads_or(any)) return;   // no row of the block is written
    amax = block_max(amax);
    if (amax == INFINITY) {               // over the finite values alone
        float finite = 0.f;
        for (long long pos = lo + r0; pos < hi; pos += kRows * rows) {
            load(pos);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float x[16];
                if (!values(i, pos + i * rows, x)) continue;
#pragma unroll
                for (int e = 0; e < 16; ++e) finite = fmaxf(finite, finite_abs(x[e]));
            }
        }
        __syncthreads();
        amax = block_max(finite);
    }
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
    // Rows are read again (from cache) unless one load held them all.
    const bool held = hi - lo <= kRows * rows;
    for (long long pos = lo + r0; pos < hi; pos += kRows * rows) {
        if (!held) load(pos);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float x[16];
            if (!values(i, pos + i * rows, x)) continue;
            uint8_t *d =
                dst + ((size_t)(row0 + (pos + i * rows - t0)) * p.kv_heads + h) * p.head_dim;
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = e4m3x4(x[4 * e] * inv, x[4 * e + 1] * inv, x[4 * e + 2] * inv,
                              x[4 * e + 3] * inv);
            *reinterpret_cast<uint2 *>(d + t.a) = make_uint2(o[0], o[1]);
            *reinterpret_cast<uint2 *>(d + t.b) = make_uint2(o[2], o[3]);
        }
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

// A call of many tokens gives a thread kFlight chunks or more of one token; a
// call of few spreads each token over more CTAs while there are SMs without one
// (64 requests x 4 proposals: 4.9 us with a CTA a token, 6.1 with three).
Spread spread(const RopeParams &p, int heads, int threads) {
    const int per = p.head_dim / 16;
    const long long chunks = (long long)heads * per, tokens = (long long)p.batch * p.k;
    Spread s{1, 1, tokens * chunks >= 152ll * 1024 * kFlight};
    if (s.many) {
        while (threads % (2 * s.per_cta) == 0 && threads / (2 * s.per_cta) % per == 0 &&
               chunks * s.per_cta < (long long)kFlight * threads)
            s.per_cta *= 2;
    } else {
        const long long full = (chunks + threads - 1) / threads;
        const long long want = (152 + tokens - 1) / tokens;
        s.splits = (int)(want < full ? want : full);
    }
    return s;
}

long long ctas(const RopeParams &p, Spread s) {
    return ((long long)p.batch * p.k + s.per_cta - 1) / s.per_cta * s.splits;
}

}  // namespace

bool rope_shape_ok(int head_dim) { return head_dim <= 1024 && cta_threads(head_dim) <= kThreads; }

cudaError_t launch_rope_append(const RopeParams &p, cudaStream_t stream) {
    const int threads = cta_threads(p.head_dim);
    const Spread s = spread(p, p.q_heads + 2 * p.kv_heads, threads);
    const long long grid = ctas(p, s);
    if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
    auto kernel = s.many ? (p.interleaved ? rope_append_kernel<true, kFlight>
                                          : rope_append_kernel<false, kFlight>)
                         : (p.interleaved ? rope_append_kernel<true, 1> : rope_append_kernel<false, 1>);
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(threads), 0, stream, p, s);
}

cudaError_t launch_rope_append_fp8(const RopeParams &p, cudaStream_t stream) {
    const int threads = cta_threads(p.head_dim);
    const Spread s = spread(p, p.q_heads, threads);
    const int blocks = (p.k + p.block_rows - 2) / p.block_rows + 1;
    const long long kv = (long long)p.batch * blocks * p.kv_heads * 2;
    const long long grid = kv + (p.q_heads > 0 ? ctas(p, s) : 0);
    if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
    auto kernel =
        s.many ? (p.interleaved ? rope_append_fp8_kernel<true, kFlight>
                                : rope_append_fp8_kernel<false, kFlight>)
               : (p.interleaved ? rope_append_fp8_kernel<true, 1> : rope_append_fp8_kernel<false, 1>);
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(threads), 0, stream, p, blocks,
                            (unsigned)kv, s);
}

}  // namespace carat
