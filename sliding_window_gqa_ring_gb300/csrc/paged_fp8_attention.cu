// paged_fp8_attention.cu -- decode / verify attention over paged e4m3 caches
// with one scale per block of tokens and KV head, on the 5th-generation
// tensor cores with 8-bit operands.
//
// For query row (j, h) of request b at position p = context_length + j, over
// the positions t in [max(0, p - window + 1), p] (log2 units throughout):
//     s_t = scale * log2(e) * ks[t] * sum_d q_d e4m3(k_td),
//     out_d = sum_t 2^(s_t - m) vs[t] e4m3(v_td) / sum_t 2^(s_t - m)
// with ks, vs the scales of the token's block.
//
// Bytes as operands.  A decode step reads each cached byte once and does few
// operations with it, so the cache has to reach the tensor core as it lies in
// memory: K and V tiles of 128 keys go from HBM through TMA into shared memory
// and from there straight into tcgen05.mma (kind::f8f6f4), with no thread
// touching them.  The other operands are split into 8-bit pieces that stand side by
// side as more columns of the same product:
//   * a query row, scaled by a power of two so its largest element lies in
//     [128, 256), is hi + lo / 16, both e4m3: four bits each and a sign make
//     up a bf16 value's eight.  That is exact down to 2^-13 of the row's largest
//     element; smaller ones are rounded to 2^-21 of it (a score that is off by
//     2^-21 of its largest products is what an fp32 sum of them gives);
//   * a weight w_t = 2^(s_t - m) vs[t] is first rounded to f16: its 2^-11 is below
//     the output's own bf16 rounding, and a third more pieces would be the price of
//     three bits more.  It then is w1 + w2 / 8 + w3 / 64, all e5m2, exactly: three
//     bits each and two signs make up f16's eleven (down to 2^-28 of the row's
//     largest weight, see kBoost).
// Keys are the M dimension of both products:
//     S^T [128 keys x 2N]  = K_tile [128 x D] . [q_hi | q_lo]^T      (K-major A)
//     O^T [128 d x 3N]    += V_tile^T [d x 128 keys] . [w1 | w2 | w3]^T (MN-major A)
// for N = 8, 16 or 32 rows; more rows (up to 128) are cut into row groups of 32.
// The scales cost nothing in the products: thread t of the softmax owns key t,
// so ks[t] is one factor of its scores, and vs[t] one of its weights.
//
// The running maximum m is that of s_t + log2 vs[t], not of s_t: it bounds the
// weights that are rounded, whatever the scales' range.  It moves only when
// exceeded by more than kSlack.  The denominator is the sum of 2^(s_t - m) itself,
// in fp32, before vs[t] and the rounding: keys with a tiny scale (a block of zero
// values) keep their share of it although their weights vanish.
//
// Range of that sum.  Scales lie in [2^-100, 2^100], so with kBoost and kSlack a
// term is at most 2^114, and the key that gave m adds at least 2^-94: terms below
// 2^-126, flushed to zero, are less than 2^-32 of it.  When m moves, by up to 200 and
// more at equal scores, 2^(old - new) itself may be below 2^-126 where its product
// with the sum is not: it is applied as two factors 2^((old - new) / 2), one after
// the other, here and in the merge.  (O may lose what lies below 2^-126 of its new
// weights.)  A thread's part of a sum (its key of every tile of a segment) stays
// below 2^127 up to 2^20 keys a segment; it is scaled by kSum = 2^-10 before the 128
// threads' parts meet, and O with it.
//
// NaN.  Keys that a row does not see get weight 0, and 0 x NaN is NaN in a product.
// So V rows outside the request's keys are zeroed in shared memory, and keys that
// some of a step's queries see and others do not are looked through for NaNs by
// warp 3; found ones are taken out of V and put into the weights of the rows that
// see them.
//
// Schedule: stream-K.  All (request, KV head) units' tiles form one sequence,
// cut into ranges of equal cost, one per CTA (with G row groups CTAs
// G r .. G r + G - 1 walk range r together, one group each, so the tiles they
// share come from L2).  A segment that covers a whole unit writes its output; the
// others leave a partial (max, sum, O) for the merge launch, which finds them
// through a table with one entry per unit.  A unit's start is charged kCharge = 5
// tiles.  Measured, 2 to 7 (us): 64 requests x 4 proposals up to 32768 keys 201, 198,
// 191, 188, 187, 187; 56 x 1 in a window of 1024 65.5, 65.5, 63.0, 62.0, 62.8, 64.0.
//
// Three launches, each started while the one before it runs (programmatic
// dependent launch): the queries' split, this kernel, the merge.
//
// Order of the launches.  Here only warp 3, which fetches the split queries, waits for
// the split launch.  The other warps read lengths, counts, page table, scales and
// pages at once: all of them were written by launches before the split, which has
// waited for those before it lets this one start.  (Every warp waiting for the whole
// split: one request of 1500 or 6005 keys 15.5 -> 16.2, 19.8 -> 21.6 us, 8 x 15
// 86.6 -> 89.7, 64 x 4 180.1 -> 182.4.)  That
// orders the writes before the reads in time; visibility is promised to a grid that
// waits, so the reads go to L2, where a finished launch's writes are, and not to an
// SM's own cache: __ldcg, and TMA, which has no other way.
//
// Warps: 0 loads tiles (TMA), 1 issues the products, 2 fetches the tiles' block
// scales ahead of the softmax, 3 fetches the split queries and looks for NaNs, 4 and
// up run the softmax: one or two groups of four warps, each with half the rows (or
// all), thread t of a group key t of the tile.  Every wait is bounded.  A wait for a
// barrier's phase is a wait for its parity, so it may only be made once the phase
// before is known to be over; a model of the roles on the CPU checks that.
//
// What it reaches (copy rate of the device: 6796 GB/s), all launches included:
// 64 requests x 4 proposals, 16/2 heads of 512, up to 32768 keys each (1044 MB):
// 180 to 184 us, 5680 to 5800 GB/s, bound by the loads but for the start, the units'
// boundaries and the merge.  56 x 1, 16/8 heads of 256, window 1024 (236 MB): 55 to 57
// us, of which about 20 do not grow with the batch (start, first loads, drain, merge;
// 224 x 1: 185 us).  8 x 15 (173 MB, 120 rows in four groups): 86 us, bound by its
// products: 32 a tile at 75 cycles each (60 at their best; their operands share
// shared memory's bandwidth with the loads) are 2400 of about 2850 cycles a tile.
// The same rows at head_dim 256 have half the products and wait for the softmax,
// 2400 cycles a tile.  One request of 1500 or 6005 keys: 15.5 and 20 us, a chain of
// latencies (split, first load to last output, merge).  One request of 32768 keys
// among 9 or 19 of 400 (16/2 heads of 512, 4 proposals): 40 us, where the same keys
// spread evenly take 29: the merge's shape goes by the average number of pieces.
#include <algorithm>
#include <atomic>

#include "carat_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tc_common.cuh"
#include "tma_host.h"

namespace carat {
namespace {

constexpr int kKeys = 128;                 // keys of a tile
constexpr int kSlab = kKeys * 128;         // bytes of 128 keys x 128 d
constexpr int kStage = 2 * kSlab;          // a stage: 128 keys x 256 d, one copy
constexpr int kSlots = 4;                  // tiles whose scales are fetched ahead
constexpr int kMaxPieces = 320;            // pieces of one unit
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kSlack = 8.f;
// Weights carry the factor 2^kBoost = kWeight: 2^(kSlack + kBoost) = 2^14 fits
// e5m2 and f16, and weights are resolved down to 2^-28 of the largest.
constexpr float kBoost = 6.f, kWeight = 64.f;
constexpr float kSum = 1.f / 1024;         // of a row's sum and O at a segment's end
// Maximum of a row that has seen no key yet: below every score, which key scales of
// 2^100 take to -1e32 and further.
constexpr float kUnset = -3e38f;

// Two shapes of CTA.  With up to 16 rows at head_dim 256 two CTAs share an SM, so
// that one streams while the other is at a unit's boundary or starting up (56
// requests x 1, window 1024: 63 us, one CTA 75); else one CTA takes the SM and its
// shared memory, with eight softmax warps (four for 8 rows; sixteen for 32 rows
// gave 101 against 100 us at 8 x 15 and 192 against 188 at 64 x 4).
// A stage is 32 KB: of 16 KB, 8 x 15 took 104 us against 95.  Tiles of 8 rows and a
// second buffer of queries where they fit: 62.7 -> 59.7 us at 56 x 1.
template <int D, int N>
struct Lay {
    static constexpr int KS = D / 128;                // 128-d blocks
    static constexpr int TS = D / 256;                // stages of a K (or V) tile
    static constexpr int OCC = D == 256 && N <= 16 ? 2 : 1;
    static constexpr int H = OCC == 2 || N == 8 ? 1 : 2;   // groups of four softmax warps
    static constexpr int NC = N / H;                  // rows of a group
    static constexpr int kSoftWarps = 4 * H, kThreads = 128 + 128 * H;
    static constexpr int PB = OCC == 2 ? 1 : 2;       // buffers of weights
    static constexpr int QB = N == 8 || (D == 256 && N == 32) ? 2 : 1;   // of queries
    static constexpr int NS = OCC == 2 ? 3 : N <= 16 ? 6 : 5;
    static constexpr int PR = (3 * N + 15) / 16 * 16; // rows of the weights' operand
    static constexpr int kCharge = 5;                 // tiles a unit's boundary costs
    static constexpr int kQBlock = 2 * N * 128;       // 128 d of the query pieces
    static constexpr int kQBytes = KS * kQBlock;
    static constexpr int kPBytes = PR * 128;          // a tile's weights
    // Weights of 32 rows lie as three pieces [128 keys][32 rows], of 8 rows as one
    // block [128 keys][w1 w2 w3 -], so a thread stores 16 bytes of its key at a time;
    // of 16 rows as [3N rows][128 keys], byte by byte (as 32 rows first were: 8 x 15
    // 96.6 us against 90.1), for want of 2 KB of shared memory.
    static constexpr bool kWide = N != 16;
    static constexpr int kOffQ = NS * kStage;
    static constexpr int kOffP = kOffQ + QB * kQBytes;
    static constexpr int kOffRed = kOffP + PB * kPBytes;
    // floats: the four key quarters' maxima or sums per row, the running
    // maxima, the rescale factors' roots, and of two segments the score factors and
    // output rows (int) of the queries
    static constexpr int kRedM = 4 * N, kRedAlpha = 5 * N, kRedQ = 6 * N;
    static constexpr int kRedFloats = 10 * N;
    static constexpr int kOffSc = kOffRed + kRedFloats * 4;      // [kSlots][2][8] scales
    static constexpr int kOffBar = kOffSc + kSlots * 64;
    static constexpr int kBars = 2 * NS + 15 + 2 * kSlots;
    static constexpr int kOffMisc = kOffBar + kBars * 8;
    static constexpr int kBytes = kOffMisc + 128;
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr int kTmemO = 4 * N;              // two S^T buffers of 2 N columns first
    static constexpr int kTmem = 4 * N + KS * PR <= 256 ? 256 : 512;
    static_assert(4 * N + KS * PR <= kTmem, "tensor memory");
    static_assert(OCC * (kAlloc + 1024) <= 233472 && kAlloc <= 232448, "shared memory");
    static_assert(OCC * kTmem <= 512, "tensor memory");
    // the softmax zeroes V rows while the tile's stages are all resident, with the
    // next tile's K in front of them
    static_assert(NS >= 2 * TS, "the ring holds a K and a V tile");
    static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kQBlock % 1024 == 0 &&
                      kPBytes % 1024 == 0, "swizzle");
    static_assert(kOffSc % 16 == 0 && kRedQ % 4 == 0 && kRedAlpha % 4 == 0, "alignment");
};

// A unit and row group's queries as the split launch leaves them: the Q operand
// as it lies in shared memory, then each row's score factor, then its row in the
// output (-1: none).
template <int D, int N>
struct Image {
    static constexpr int kOperand = D / 128 * 2 * N * 128;
    static constexpr int kBytes = kOperand + 2 * N * 4;
};

struct Plan {
    uint8_t *images;    // [B * Hkv * groups] Image
    int groups;     // row groups of a unit
    int ranges;     // ranges of the tile sequence (grid = ranges * groups)
    float2 *part_ml;    // [2 * grid][N] (max, sum)
    float *part_o;      // [2 * grid][N][D]
    // per (request, KV head, row group): range of the first piece and its slot
    // (-1: whole, nothing to merge), range of the last piece
    int2 *first;
    int *last;
};

// One request of the call: its tokens before this step and its queries.
struct Request {
    int ctx, n;
};

// (through L2: see "Order of the launches")
__device__ __forceinline__ Request load_request(const PagedFp8Params &p, int b) {
    return {__ldcg(p.context_lengths + b), p.new_counts ? __ldcg(p.new_counts + b) : p.k};
}

__device__ __forceinline__ bool request_ok(const PagedFp8Params &p, Request r) {
    return r.ctx >= 0 && r.n >= 0 && r.n <= p.k && r.n <= p.capacity - r.ctx;
}

// Tiles of a request: [first, first + count) of its 128-position tiles; 0 when it
// has no queries or is rejected.
__device__ __forceinline__ int request_tiles(const PagedFp8Params &p, Request r, int *first) {
    *first = 0;
    if (!request_ok(p, r) || r.n == 0) return 0;
    if (p.window > 0 && r.ctx >= p.window) *first = (r.ctx - p.window + 1) / kKeys;
    return (r.ctx + (r.n - 1)) / kKeys - *first + 1;
}

// What a CTA's roles share besides the barriers.
struct Shared {
    uint32_t tmem;
    int abort_flag;
    int b0, c0, off0;       // first segment: request, KV head, tiles of the unit before it
    int s, e;               // the CTA's tiles of the sequence
    int nans[2];            // of two segments: NaNs among values that not every query sees
};

struct Segment {
    int b, c, ctx, n;
    int first, ntiles;      // the unit's tiles
    int x0, x1;             // those of this segment
    bool opens;             // the segment opens the CTA's range
};

// Walks a CTA's range as segments, one per unit it touches.
struct SegIter {
    Request rq;
    int pos, end, start, b, c, off, first, ntiles;

    __device__ void init(const PagedFp8Params &p, const volatile Shared *sh) {
        pos = start = sh->s;
        end = sh->e;
        b = sh->b0;
        c = sh->c0;
        off = sh->off0;
        ntiles = 0;
        if (pos < end) {
            rq = load_request(p, b);
            ntiles = request_tiles(p, rq, &first);
        }
    }

    // To the next unit that has tiles.
    __device__ void advance(const PagedFp8Params &p) {
        off = 0;
        if (++c < p.kv_heads) return;
        c = 0;
        ntiles = 0;
        while (ntiles == 0 && b + 1 < p.batch) {
            ++b;
            rq = load_request(p, b);
            ntiles = request_tiles(p, rq, &first);
        }
    }

    __device__ __noinline__ bool next(const PagedFp8Params &p, Segment &sg) {
        if (pos >= end || off >= ntiles) return false;
        const int len = min(ntiles - off, end - pos);
        sg.b = b;
        sg.c = c;
        sg.ctx = rq.ctx;
        sg.n = rq.n;
        sg.first = first;
        sg.ntiles = ntiles;
        sg.x0 = off;
        sg.x1 = off + len;
        sg.opens = pos == start;
        pos += len;
        off += len;
        if (off == ntiles && pos < end) advance(p);
        return true;
    }
};

// Warp 0: this CTA's range.  A unit costs its tiles and kCharge more (its
// segment boundary: a new Q, an output or partial); tile o of the unit that
// begins at cost U sits at U + charge + o, and tile t belongs to range
// floor(cost(t) / len).  A call with fewer tiles than ranges charges nothing,
// and every tile has a range to itself.  The requests' tile counts are read
// once, four loads of a lane in flight, and kept in `held` (room for `room`
// of them) for the second pass.
__device__ __noinline__ void locate_range(const PagedFp8Params &p, int ranges, int rix, int lane,
                                          int unit_charge, int *held, int room, Shared *sh) {
    int tiles = 0, units = 0;
#pragma unroll 1
    for (int base = 0; base < p.batch; base += 128) {
        Request rq[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = base + 32 * i + lane;
            rq[i] = b < p.batch ? load_request(p, b) : Request{-1, 0};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = base + 32 * i + lane;
            int first;
            const int v = request_tiles(p, rq[i], &first);
            tiles += v;
            units += v > 0 ? 1 : 0;
            if (b < p.batch && b < room) held[b] = v;
        }
    }
    __syncwarp();
    tiles = __reduce_add_sync(kFull, tiles) * p.kv_heads;
    units = __reduce_add_sync(kFull, units) * p.kv_heads;
    const int charge = tiles >= ranges ? unit_charge : 0;
    const int cost = tiles + charge * units;
    int len = (cost + ranges - 1) / ranges;
    if (len < charge + 1) len = charge + 1;
    // The first tiles at cost positions >= X0 and >= X1 (none: `tiles`).
    const int X0 = rix * len, X1 = rix + 1 < ranges ? X0 + len : cost;
    int at0 = tiles, at1 = tiles, b0 = 0, c0 = 0, off0 = 0;
    int cum_cost = 0, cum_tiles = 0;
#pragma unroll 1
    for (int base = 0; base < p.batch && cum_cost <= X1; base += 32) {
        const int b = base + lane;
        int v = 0, first;
        if (b < p.batch) v = b < room ? held[b] : request_tiles(p, load_request(p, b), &first);
        const int per = v + charge;
        const int vc = v > 0 ? p.kv_heads * per : 0, vt = p.kv_heads * v;
        int ic = vc, it = vt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yc = __shfl_up_sync(kFull, ic, o), yt = __shfl_up_sync(kFull, it, o);
            if (lane >= o) ic += yc, it += yt;
        }
        const int lo = cum_cost + ic - vc, tlo = cum_tiles + it - vt;
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int X = which ? X1 : X0;
            const bool mine = vc > 0 && X >= lo && X < lo + vc;
            const unsigned hit = __ballot_sync(kFull, mine);
            if (!hit) continue;
            const int src = __ffs(hit) - 1;
            int at = 0, j = 0, o = 0;
            if (mine) {
                j = (X - lo) / per;
                const int r = X - lo - j * per;
                o = r <= charge ? 0 : r - charge;
                at = tlo + j * v + o;
            }
            at = __shfl_sync(kFull, at, src);
            if (which) {
                at1 = at;
            } else {
                at0 = at;
                b0 = base + src;
                c0 = __shfl_sync(kFull, j, src);
                off0 = __shfl_sync(kFull, o, src);
            }
        }
        cum_cost += __shfl_sync(kFull, ic, 31);
        cum_tiles += __shfl_sync(kFull, it, 31);
    }
    if (lane == 0) {
        sh->s = at0;
        sh->e = at1;
        sh->b0 = b0;
        sh->c0 = c0;
        sh->off0 = off0;
    }
    __syncwarp();
}

// Wait for a barrier phase; false after two seconds, or when another role gave
// up (which is recorded and reported once).  The polling is out of line: the
// roles' loops share one small instruction cache.
__device__ __noinline__ bool await_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                        int *dev_status) {
    const uint64_t t0 = tc::globaltimer_ns();
    for (uint32_t round = 1;; ++round) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (tc::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (tc::wait_expired(t0, round, 2000000000ull)) {
            *abort_flag = 1;
            set_status(dev_status, CARAT_DEV_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool await(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                      int *dev_status) {
    return tc::mbar_try_wait(bar, parity) || await_slow(bar, parity, abort_flag, dev_status);
}

// Barrier of the 128 threads of one group of softmax warps (of H); true when any
// of them says so.
template <int H>
__device__ __forceinline__ bool half_any(int half, bool pred) {
    uint32_t out;
    if constexpr (H == 1) {
        asm volatile(
            "{\n\t.reg .pred pin, pout;\n\t"
            "setp.ne.u32 pin, %1, 0;\n\t"
            "bar.red.or.pred pout, 1, 128, pin;\n\t"
            "selp.u32 %0, 1, 0, pout;\n\t}"
            : "=r"(out)
            : "r"((uint32_t)pred)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred pin, pout;\n\t"
            "setp.ne.u32 pin, %1, 0;\n\t"
            "bar.red.or.pred pout, %2, 128, pin;\n\t"
            "selp.u32 %0, 1, 0, pout;\n\t}"
            : "=r"(out)
            : "r"((uint32_t)pred), "r"(half + 1)
            : "memory");
    }
    return out != 0;
}

// v[i] is this lane's value of row i; returns the row this lane ends up with,
// whose reduction over the 32 lanes is then v[0].
template <int NC, bool kMax>
__device__ __forceinline__ int transpose_reduce(float (&v)[NC], int lane) {
    int row = 0;
#pragma unroll
    for (int s = 0; s < 5; ++s) {
        const int off = 16 >> s, cnt = (NC >> s) > 1 ? (NC >> s) : 1;
        const bool upper = (lane & off) != 0;
        if (cnt >= 2) {
            const int h = cnt / 2;
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const float send = upper ? v[i] : v[i + h], keep = upper ? v[i + h] : v[i];
                const float got = __shfl_xor_sync(kFull, send, off);
                v[i] = kMax ? fmaxf(keep, got) : keep + got;
            }
            if (upper) row += h;
        } else {
            const float got = __shfl_xor_sync(kFull, v[0], off);
            v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
        }
    }
    return row;
}

template <int NC>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[NC]) {
    if constexpr (NC == 16) tc::tmem_ld16(addr, r);
    else tc::tmem_ld8(addr, r);
}

template <int NC>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[NC]) {
    if constexpr (NC == 16) tc::tmem_st16(addr, r);
    else tc::tmem_st8(addr, r);
}

// Two fp32 values in one register pair, for the packed instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint32_t low_mask(int n) { return n >= 32 ? kFull : (1u << n) - 1u; }

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t b) {
    uint32_t h;
    asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
        : "=r"(h)
        : "r"(b));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Two f16 values -> their nearest e5m2 bytes (first in the low one).
__device__ __forceinline__ uint32_t e5m2x2(__half2 h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;"
        : "=h"(r)
        : "r"(*reinterpret_cast<const uint32_t *>(&h)));
    return r;
}

// e5m2 is f16's upper byte.
__device__ __forceinline__ __half2 e5m2x2_to_f16x2(uint32_t b) {
    const uint32_t w = __byte_perm(b, 0, 0x1404);
    return *reinterpret_cast<const __half2 *>(&w);
}

// One query row into the two pieces' rows of the Q operand (row r and N + r of
// every 128-d block), by one warp.  Returns the factor that takes the power
// of two out of the scores again (NaN for a row that is not finite, 0 for none).
template <int D, int N>
__device__ __forceinline__ float split_query(uint8_t *s_q, const uint16_t *row, int r, int lane) {
    constexpr int E = D / 32;   // 16 or 8 elements of a lane
    uint32_t w[E / 2];
    uint32_t top = 0;           // largest |q|, as bits
    if (row) {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(row + lane * E)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            top = max(top, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) w[i] = 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    int s = 7 - ((int)(top >> 23) - 127);
    // Zero and tiny rows.  Up to 2^120 the factor 2^-s and the score factor formed from
    // it stay normal numbers, and a row of 2^-126 still has bf16's eight bits; what
    // is lost below is less than 2^-15 of the softmax scale in any score, whatever the
    // key scales.
    s = min(s, 120);
    const float up = __int_as_float((127 + s) << 23);
    uint32_t hi[E / 4], lo[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        uint32_t h2[2], l2[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const float a = bf16lo(w[2 * i + z]) * up, b = bf16hi(w[2 * i + z]) * up;
            h2[z] = e4m3x2(a, b);
            const float2 f = e4m3x2_to_f32(h2[z]);
            l2[z] = e4m3x2((a - f.x) * 16.f, (b - f.y) * 16.f);
        }
        hi[i] = h2[0] | (h2[1] << 16);
        lo[i] = l2[0] | (l2[1] << 16);
    }
    uint8_t *block = s_q + (lane * E / 128) * (2 * N * 128);
    const int byte = lane * E % 128, chunk = byte / 16;
    uint8_t *ph = block + r * 128 + ((chunk ^ (r & 7)) << 4) + byte % 16;
    uint8_t *pl = ph + N * 128;   // N is a multiple of 8: the same swizzle
    if constexpr (E == 16) {
        *reinterpret_cast<uint4 *>(ph) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(pl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    } else {
        *reinterpret_cast<uint2 *>(ph) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2 *>(pl) = make_uint2(lo[0], lo[1]);
    }
    if (!row) return 0.f;
    return top >= 0x7f800000u ? __int_as_float(0x7fc00000) : __int_as_float((127 - s) << 23);
}

// Which bytes of a word of e4m3 are NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// A key that some of the request's queries see and others do not is one of
// [ctx + 1, keys), or with a window one of [lowest, keys - window).  A warp looks
// through the value bytes of such keys in a segment for NaNs.
template <int D>
__device__ __noinline__ bool some_nan(const PagedFp8Params &p, const Segment &sg, int lane) {
    constexpr int kChunks = D / 16;
    const int keys = sg.ctx + sg.n, begin = (sg.first + sg.x0) * kKeys;
    const int end = min(keys, begin + (sg.x1 - sg.x0 - 1) * kKeys + kKeys);
    const int lowest = p.window > 0 && sg.ctx >= p.window ? sg.ctx - p.window + 1 : 0;
    const int a0 = max(sg.ctx + 1, begin), na = max(end - a0, 0);
    const int b0 = max(lowest, begin);
    const int nb = p.window > 0 ? max(min(keys - p.window, end) - b0, 0) : 0;
    uint32_t found = 0;
#pragma unroll 4
    for (int i = lane; i < (na + nb) * kChunks; i += 32) {
        const int key = i / kChunks, pos = key < na ? a0 + key : b0 + key - na;
        const long long row =
            paged_row(p.page_table, p.max_pages, p.page_rows, p.num_pages, sg.b, pos);
        if (row < 0) continue;
        const uint4 w = *reinterpret_cast<const uint4 *>(
            p.v_pages + ((size_t)row * p.kv_heads + sg.c) * D + i % kChunks * 16);
        found |= nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w);
    }
    return __any_sync(kFull, found != 0);
}

// Replaces the NaNs in the V row of a tile's key t by negative zeros; whether it has
// any.  The tile's V lies in ring slots base, base + 1, ...  The bytes come from the
// page: the other group of softmax warps may have replaced them already.
template <int D, int NS>
__device__ __noinline__ bool remove_nans(const PagedFp8Params &p, uint8_t *smem, uint32_t base,
                                         int t, int b, int c, int pos) {
    const long long row = paged_row(p.page_table, p.max_pages, p.page_rows, p.num_pages, b, pos);
    if (row < 0) return false;
    const uint8_t *src = p.v_pages + ((size_t)row * p.kv_heads + c) * D;
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < D / 4; ++i) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(src)[i], nan = nan_bytes(w);
        if (!nan) continue;
        any = true;
        const int chunk = i / 4;
        *reinterpret_cast<uint32_t *>(smem + (base + chunk / 16) % NS * kStage +
                                      chunk / 8 % 2 * kSlab + t * 128 +
                                      ((chunk ^ t) & 7) * 16 + i % 4 * 4) =
            (w & ~nan) | (nan & 0x80808080u);
    }
    return any;
}

// The queries of every unit and row group as 8-bit pieces (Image), and NaN outputs
// for the requests that are rejected on the device.  One CTA per unit and row
// group, one warp per row.  It runs ahead of the attention, which starts
// loading keys meanwhile: there each CTA fetches an image with one copy when it
// comes to the unit, where splitting rows in place took the softmax 5000 to 8000
// cycles at every unit's start.
template <int D, int N>
__global__ void __launch_bounds__(32 * N) paged_fp8_split_kernel(
    const __grid_constant__ PagedFp8Params p, const Plan plan) {
    // In this order: the attention reads what the launches before this one wrote
    // without waiting itself (see "Order of the launches").
    wait_for_prior_launch();
    let_next_launch_start();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int u = blockIdx.x, rg = u % plan.groups, bc = u / plan.groups;
    const int b = bc / p.kv_heads, c = bc % p.kv_heads;
    const Request rq = load_request(p, b);
    const bool ok = request_ok(p, rq);
    if (!ok && threadIdx.x == 0 && c == 0 && rg == 0) set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
    uint8_t *image = plan.images + (size_t)u * Image<D, N>::kBytes;
    float *factor = reinterpret_cast<float *>(image + Image<D, N>::kOperand);
    int *out_row = reinterpret_cast<int *>(factor + N);
    const int r = warp, ur = rg * N + r, j = ur / p.group;
    int at = ur < p.group * p.k
                 ? (b * p.k + j) * p.q_heads + c * p.group + ur - j * p.group
                 : -1;
    if (!ok) {
        if (at >= 0)
            for (int i = lane; i < D / 2; i += 32)
                reinterpret_cast<uint32_t *>(p.out + (size_t)at * D)[i] = 0x7fc07fc0u;
        return;
    }
    if (j >= rq.n) at = -1;   // a query behind the request's last
    const float f = split_query<D, N>(image, at >= 0 ? p.q + (size_t)at * D : nullptr, r, lane);
    if (lane == 0) {
        factor[r] = f * p.scale_log2;
        out_row[r] = at;
    }
}

template <int D, int N>
__global__ void __launch_bounds__(Lay<D, N>::kThreads, Lay<D, N>::OCC)
    paged_fp8_kernel(const __grid_constant__ PagedFp8Params p, const Plan plan,
                     const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v) {
    using L = Lay<D, N>;
    constexpr int KS = L::KS, TS = L::TS, NS = L::NS, NC = L::NC;
    constexpr int kSoftWarps = L::kSoftWarps, kThreads = L::kThreads;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rix = blockIdx.x / plan.groups, rg = blockIdx.x % plan.groups;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    uint64_t *empty = full + NS;
    uint64_t *s_full = empty + NS;      // [2] scores of a tile ready
    uint64_t *p_full = s_full + 2;      // [2] weights of a tile written
    uint64_t *o_done = s_full + 4;      // [2] PV product of a tile done
    uint64_t *q_full = s_full + 6;      // [2] queries of a segment landed
    uint64_t *q_empty = s_full + 8;     // [2] last QK product of a segment done
    uint64_t *q_free = s_full + 10;     // [2] factors of a segment's queries used
    uint64_t *fin = s_full + 12;
    uint64_t *nan_full = s_full + 13;   // [2] a segment looked through for NaNs
    uint64_t *sc_full = s_full + 15;    // [kSlots] scales of a tile fetched
    uint64_t *sc_empty = sc_full + kSlots;
    uint8_t *s_q = smem + L::kOffQ;
    uint8_t *s_p = smem + L::kOffP;
    float *red = reinterpret_cast<float *>(smem + L::kOffRed);
    float *s_sc = reinterpret_cast<float *>(smem + L::kOffSc);
    Shared *sh = reinterpret_cast<Shared *>(smem + L::kOffMisc);
    volatile int *abort_flag = &sh->abort_flag;
    int *status = p.dev_status;

    // the merge launch may start once every CTA of this grid runs (it waits for this one
    // before it touches memory, and the next call's split for the merge)
    if (threadIdx.x == 0) let_next_launch_start();

    // Pool row of a tile's first position; -1 for a page outside the pool.
    const int pages_shift_tiles = p.page_rows / kKeys;   // tiles of a page
    auto tile_row = [&](int page, int tile) -> long long {
        if (page < 0 || page >= p.num_pages) return -1;
        return (long long)page * p.page_rows + (long long)(tile % pages_shift_tiles) * kKeys;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ tiles
        if (lane == 0) {
            tc::tma_prefetch_map(&map_k);
            tc::tma_prefetch_map(&map_v);
            for (int i = 0; i < NS; ++i) {
                tc::mbar_init(&full[i], 1);
                tc::mbar_init(&empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&s_full[i], 1);
                tc::mbar_init(&p_full[i], kSoftWarps);
                tc::mbar_init(&o_done[i], 1);
                tc::mbar_init(&q_full[i], 1);
                tc::mbar_init(&nan_full[i], 1);
                tc::mbar_init(&q_free[i], kSoftWarps);
                tc::mbar_init(&q_empty[i], 1);
            }
            tc::mbar_init(fin, 1);
            for (int i = 0; i < kSlots; ++i) {
                tc::mbar_init(&sc_full[i], 1);
                tc::mbar_init(&sc_empty[i], kSoftWarps);
            }
            sh->abort_flag = 0;
            tc::fence_mbar_init();
        }
        locate_range(p, plan.ranges, rix, lane, L::kCharge, reinterpret_cast<int *>(s_p),
                     L::PB * L::kPBytes / 4, sh);
        __threadfence_block();
        __syncwarp();
        // the others wait for this; the loads need not wait for them
        asm volatile("bar.arrive 3, %0;" ::"n"(kThreads) : "memory");
        if (lane == 0) {
            // K and V rows are read once, unless row groups share them
            const uint64_t pol = plan.groups > 1 ? tc::l2_evict_normal_policy()
                                                 : tc::l2_evict_first_policy();
            SegIter it;
            it.init(p, sh);
            Segment sg, nx;
            bool have = it.next(p, sg), have_next = false;
            int pi = -1, page = 0, pi_next = -1, page_next = 0;   // a page read ahead
            auto read_ahead = [&](const Segment &to, int want) {
                pi_next = want < p.max_pages ? want : -1;
                if (pi_next >= 0) page_next = __ldcg(p.page_table + (size_t)to.b * p.max_pages + want);
            };
            uint32_t cnt = 0;
            bool alive = true;
            auto issue = [&](const CUtensorMap *map, long long row, int c) {
                for (int ks = 0; ks < TS && alive; ++ks) {
                    const int s = cnt % NS;
                    if (cnt >= NS &&
                        !await(&empty[s], ((cnt / NS) & 1) ^ 1, abort_flag, status)) {
                        alive = false;
                        return;
                    }
                    tc::mbar_arrive_expect_tx(&full[s], kStage);
                    tc::tma_load_4d(smem + s * kStage, map, 0, (int)row, 2 * ks, c, &full[s], pol);
                    ++cnt;
                }
            };
            while (have && alive) {
                long long row = 0, prev_row = 0;
                // K of a tile before V of the one in front of it
                for (int x = sg.x0; x <= sg.x1 && alive; ++x) {
                    prev_row = row;
                    if (x < sg.x1) {
                        const int tile = sg.first + x, want = tile / pages_shift_tiles;
                        if (want != pi) {
                            if (want != pi_next) read_ahead(sg, want);
                            page = page_next;
                            pi = want;
                            read_ahead(sg, want + 1);
                        }
                        row = tile_row(page, tile);
                        if (row < 0) {   // loads the zero fill past the pool's end
                            set_status(status, CARAT_DEV_BAD_CACHE_ID);
                            row = (long long)p.num_pages * p.page_rows;
                        }
                        issue(&map_k, row, sg.c);
                    }
                    if (x > sg.x0) issue(&map_v, prev_row, sg.c);
                    // The next segment is looked up early, with the ring full: its code and
                    // data come late from a memory system that is kept busy (at the last
                    // tile, the ring ran empty for 3 to 6 us: 64 x 4 184.5 us against 182.3).
                    if (x == sg.x0 + 1) have_next = it.next(p, nx);
                }
                have = have_next;
                sg = nx;
                pi = -1;
                if (have) read_ahead(sg, (sg.first + sg.x0) / pages_shift_tiles);
            }
            // the last copies land before the CTA goes, whichever role stops early
            for (uint32_t i = cnt > (uint32_t)NS ? cnt - NS : 0; i < cnt; ++i)
                tc::mbar_wait(&full[i % NS], (i / NS) & 1, 100000000ull);
        }
        __syncwarp();
    } else {
        if (warp == 1) {
            tc::tmem_alloc(&sh->tmem, L::kTmem);
            tc::tmem_relinquish();
        }
        tc::tc_fence_before();
        asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory");
        tc::tc_fence_after();
    }

    if (warp == 1) {
        // ------------------------------------------------------------ products
        constexpr uint32_t idesc_qk = tc::idesc_e4m3_f32(128, 2 * N, false, false);
        constexpr uint32_t idesc_pv = tc::idesc_e4m3_f32(128, L::PR, true, true, L::kWide);
        const uint32_t tmem = sh->tmem;
        // descriptors in units of 16 bytes of shared memory: 32 elements along K
        // are 2 units in a K-major operand, 32 rows of 128 bytes in V
        const uint64_t k_desc = tc::sdesc_sw128(tc::smem_u32(smem), 16, 1024);
        const uint64_t v_desc = tc::sdesc_sw128(tc::smem_u32(smem), kSlab, 1024);
        const uint64_t q_desc = tc::sdesc_sw128(tc::smem_u32(s_q), 16, 1024);
        const uint64_t p_desc = L::kWide ? tc::sdesc_sw32(tc::smem_u32(s_p), kKeys * 32, 256)
                                         : tc::sdesc_sw128(tc::smem_u32(s_p), 16, 1024);
        constexpr int kPStep = L::kWide ? 64 : 2;   // 32 keys of the weights
        SegIter it;
        it.init(p, sh);
        Segment sg, nx;
        bool alive = true, have = it.next(p, sg);
        uint32_t g = 0;                 // tiles before this segment
        int ms = 0;                     // the next stage and its phase
        uint32_t mphase = 0;
        auto advance = [&]() {
            if (++ms == NS) {
                ms = 0;
                mphase ^= 1;
            }
        };
        // the warp stays together: one lane issues, all hold the operands
        auto wait_all = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(kFull, await(bar, parity, abort_flag, status)) != 0;
        };
        // In the loads' order: QK of a tile before PV of the one in front of it.
        for (int si = 0; have && alive; ++si) {
            alive = wait_all(&q_full[si & 1], (si >> 1) & 1);
            const int n = sg.x1 - sg.x0;
            bool have_next = false;
#pragma unroll 1
            for (int x = 0; x <= n && alive; ++x) {
                if (x < n) {
                    // S^T[y & 1] = K . [q_hi | q_lo]^T
                    const uint32_t y = g + x, d = tmem + (y & 1) * 2 * N;
                    uint64_t q = q_desc + si % L::QB * (L::kQBytes / 16);
#pragma unroll 1
                    for (int ks = 0; ks < TS; ++ks) {
                        if (!(alive = wait_all(&full[ms], mphase))) break;
                        tc::tc_fence_after();
                        const uint64_t a = k_desc + (uint32_t)ms * (kStage / 16);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_f8_ss_warp(d, a + kk / 4 * (kSlab / 16) + 2 * (kk % 4),
                                               q + kk / 4 * (L::kQBlock / 16) + 2 * (kk % 4), idesc_qk,
                                               (ks | kk) != 0);
                        tc::mma_commit_warp(&empty[ms]);
                        q += 2 * L::kQBlock / 16;
                        advance();
                    }
                    if (!alive) break;
                    tc::mma_commit_warp(&s_full[y & 1]);
                    if (x + 1 == n) tc::mma_commit_warp(&q_empty[si & 1]);
                    if (x == 0) have_next = it.next(p, nx);   // early, as the loads do
                }
                if (x > 0) {
                    // O^T += V^T . [w1 | w2 | w3]^T of the tile before
                    const uint32_t h = g + x - 1;
                    if (!(alive = wait_all(&p_full[h & 1], (h >> 1) & 1))) break;
                    tc::tc_fence_after();
                    const uint64_t w = p_desc + h % L::PB * (L::kPBytes / 16);
                    uint32_t d = tmem + L::kTmemO;
#pragma unroll 1
                    for (int vs = 0; vs < TS; ++vs) {
                        if (!(alive = wait_all(&full[ms], mphase))) break;
                        tc::tc_fence_after();
                        const uint64_t a = v_desc + (uint32_t)ms * (kStage / 16);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_f8_ss_warp(d + kk / 4 * L::PR,
                                               a + kk / 4 * (kSlab / 16) + 256 * (kk % 4),
                                               w + kPStep * (kk % 4), idesc_pv,
                                               !(x == 1 && kk % 4 == 0));
                        tc::mma_commit_warp(&empty[ms]);
                        d += 2 * L::PR;
                        advance();
                    }
                    if (!alive) break;
                    tc::mma_commit_warp(&o_done[h & 1]);
                }
            }
            g += n;
            have = have_next;
            sg = nx;
        }
        // so do the last products
        tc::mma_commit_warp(fin);
        tc::mbar_wait(fin, 0, 100000000ull);
    } else if (warp == 2) {
        // ------------------------------------------------------------ scales
        // Two tiles at a time: lanes 0-7 the K scales and 8-15 the V scales of
        // the first tile's (up to) eight blocks, lanes 16-31 those of the second.
        SegIter it;
        it.init(p, sh);
        Segment sg, nx;
        bool alive = true, have = it.next(p, sg);
        const int blocks = kKeys / p.block_rows, i = lane & 7;
        const float *src = (lane & 8) ? p.v_scales : p.k_scales;
        uint32_t g = 0;
        while (have && alive) {
            bool have_next = false;
            for (int x = sg.x0; x < sg.x1 && alive; x += 2) {
                const int n = min(sg.x1 - x, 2), tile = sg.first + x + lane / 16;
                float v = 1.f;   // a page outside the pool: K and V are zeros, any scale will do
                if (lane / 16 < n && i < blocks) {
                    const int page = __ldcg(p.page_table + (size_t)sg.b * p.max_pages +
                                            tile / pages_shift_tiles);
                    const long long row = tile_row(page, tile);
                    if (row >= 0)
                        v = __ldcg(src + (size_t)(row / p.block_rows + i) * p.kv_heads + sg.c);
                }
                for (int z = 0; z < n; ++z, ++g) {
                    const int slot = g % kSlots;
                    alive = alive && (g < kSlots || await(&sc_empty[slot], ((g / kSlots) & 1) ^ 1,
                                                          abort_flag, status));
                    alive = __all_sync(kFull, alive);
                    if (!alive) break;
                    if (lane / 16 == z) s_sc[slot * 16 + (lane & 15)] = v;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sc_full[slot]);
                }
                if (x == sg.x0) have_next = it.next(p, nx);
            }
            have = have_next;
            sg = nx;
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ queries
        // Each segment's queries as the split launch left them, once the last QK
        // product of the segment whose buffer they take has read its own.
        wait_for_prior_launch();
        SegIter it;
        it.init(p, sh);
        Segment sg;
        int si = 0;
        for (; it.next(p, sg); ++si) {
            bool alive = true;
            if (lane == 0) {
                const int was = si - L::QB;   // the segment whose buffer this one takes
                alive = (was < 0 || await(&q_empty[was & 1], (was >> 1) & 1, abort_flag, status)) &&
                        (si < 2 || await(&q_free[si & 1], ((si - 2) >> 1) & 1, abort_flag, status));
                if (alive) {
                    const uint8_t *image =
                        plan.images + (((size_t)sg.b * p.kv_heads + sg.c) * plan.groups + rg) *
                                          Image<D, N>::kBytes;
                    tc::mbar_arrive_expect_tx(&q_full[si & 1], Image<D, N>::kBytes);
                    tc::bulk_load(s_q + si % L::QB * L::kQBytes, image, Image<D, N>::kOperand,
                                  &q_full[si & 1]);
                    tc::bulk_load(red + L::kRedQ + (si & 1) * 2 * N, image + Image<D, N>::kOperand,
                                  2 * N * 4, &q_full[si & 1]);
                }
            }
            if (!__all_sync(kFull, alive)) break;
            const bool any = sg.n > 1 && some_nan<D>(p, sg, lane);
            if (lane == 0) {
                sh->nans[si & 1] = any;
                tc::mbar_arrive(&nan_full[si & 1]);
            }
        }
        for (int i = si > 2 ? si - 2 : 0; i < si; ++i)   // the last copies land
            tc::mbar_wait(&q_full[i & 1], (i >> 1) & 1, 100000000ull);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax
        const int half = L::H == 1 ? 0 : (warp - 4) / 4, q4 = warp & 3;
        const int t = q4 * 32 + lane;                  // key of the tile, or d of an O block
        const uint32_t tmem = sh->tmem;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const int r0 = half * NC;                      // first row of this half
        const int row0 = rg * N;                       // first of the unit's rows in this group
        const int block = t / p.block_rows;
        float *red_max = red, *s_m = red + L::kRedM, *s_alpha = red + L::kRedAlpha;

        SegIter it;
        it.init(p, sh);
        Segment sg, nx;
        bool alive = true, have = it.next(p, sg);
        int si = 0;
        uint32_t g = 0;
        while (have && alive) {
            // the next segment is looked up early, behind the first tile
            bool have_next = sg.x1 - sg.x0 == 1 && it.next(p, nx);
            const bool whole = sg.x0 == 0 && sg.x1 == sg.ntiles;
            if (half == 0 && t == 0) {
                const size_t u = ((size_t)sg.b * p.kv_heads + sg.c) * plan.groups + rg;
                if (sg.x0 == 0) plan.first[u] = make_int2(rix, whole ? -1 : sg.opens ? 0 : 1);
                if (sg.x1 == sg.ntiles) plan.last[u] = rix;
            }
            // (copies: what its address is taken of is read from memory again and again)
            const int x0 = sg.x0, x1 = sg.x1, ctx = sg.ctx, nq = sg.n, from = sg.first * kKeys;
            // first key of query 0, and the keys' end
            const int lowest = p.window > 0 && ctx >= p.window ? ctx - p.window + 1 : 0;
            const int keys = ctx + nq;
            const int rows_here = min(N, p.group * nq - row0);
            // nm: kBoost - running maximum of each row (0 while it has none)
            float nm[NC], l[NC];
#pragma unroll
            for (int e = 0; e < NC; ++e) nm[e] = 0.f, l[e] = 0.f;
            bool unset = true;   // some row has no maximum yet
            // Rows of this half that see the key at a position: query j does when
            // ctx + j >= pos > ctx + j - window.
            auto seen_rows = [&](int pos) -> uint32_t {
                const int dj = pos - ctx;
                const int jlo = max(dj, 0);
                const int jhi = p.window > 0 && dj < nq - p.window ? dj + p.window : nq;
                const int lo = min(max(jlo * p.group - row0 - r0, 0), NC);
                const int hi = min(max(min(jhi * p.group - row0, rows_here) - r0, 0), NC);
                return low_mask(hi) & ~low_mask(lo);
            };
            const float *qs = red + L::kRedQ + (si & 1) * 2 * N + r0;
            const int *out_row = reinterpret_cast<const int *>(qs) + N;
            alive = __all_sync(kFull, await(&q_full[si & 1], (si >> 1) & 1, abort_flag, status));
            for (int x = x0; x < x1; ++x, ++g) {
                const bool first = x == x0;
                const int slot = g % kSlots;
                const bool ok = __all_sync(
                    kFull, alive && await(&sc_full[slot], (g / kSlots) & 1, abort_flag, status) &&
                               await(&s_full[g & 1], (g >> 1) & 1, abort_flag, status));
                const int t0 = from + x * kKeys, pos = t0 + t;
                const bool data = pos >= lowest && pos < keys;
                float ks = 0.f, vs = 1.f;
                if (ok) {
                    tc::tc_fence_after();
                    ks = s_sc[slot * 16 + block];
                    // (a block without keys may have any scale)
                    if (data) vs = s_sc[slot * 16 + 8 + block];
                }
                __syncwarp();
                if (ok && lane == 0) tc::mbar_arrive(&sc_empty[slot]);
                // d = score - maximum + kBoost: 2^d is the key's part of the sum, and
                // 2^d vs, at most 2^(kSlack + kBoost), its weight
                float lv = __log2f(vs);   // (a bound: any value near will do)
                float d[NC];
                if (ok) {
                    uint32_t h[NC], w[NC];
                    const uint32_t at = tmem + (g & 1) * 2 * N + lanes + r0;
                    tmem_load<NC>(at, h);
                    tmem_load<NC>(at + N, w);
                    const uint64_t ks2 = pack2(ks, ks);
                    const uint64_t lo2 = pack2(0.0625f, 0.0625f);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < NC; e += 2) {
                        const uint64_t q2 = *reinterpret_cast<const uint64_t *>(qs + e);
                        const uint64_t s2 = fma2(pack2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])),
                                                 lo2, pack2(__uint_as_float(h[e]), __uint_as_float(h[e + 1])));
                        unpack2(fma2(s2, mul2(ks2, q2), pack2(nm[e], nm[e + 1])), d[e], d[e + 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < NC; ++e) d[e] = -INFINITY;
                }
                // A tile that not every row sees whole: mask by position.
                const bool edge = t0 + kKeys - 1 > ctx ||
                                  (p.window > 0 && t0 <= keys - 1 - p.window);
                if (edge) {
                    const uint32_t seen = data ? seen_rows(pos) : 0u;
                    // rows that see a key without a scale are NaN, the others not
                    const bool bad = !(vs > 0.f && vs < INFINITY);
                    if (bad) vs = 1.f, lv = 0.f;
#pragma unroll
                    for (int e = 0; e < NC; ++e) {
                        if (bad) d[e] = __int_as_float(0x7fc00000);
                        if (!((seen >> e) & 1u)) d[e] = -INFINITY;
                    }
                }
                float top = d[0];
#pragma unroll
                for (int e = 1; e < NC; ++e) top = fmaxf(top, d[e]);
                bool rescale = false;
                if (half_any<L::H>(half, unset || edge || top > kSlack + kBoost - lv || !ok || *abort_flag)) {
                    float y[NC];
#pragma unroll
                    for (int e = 0; e < NC; ++e) {
                        d[e] -= nm[e];
                        y[e] = d[e] + lv;
                    }
                    const int rr = transpose_reduce<NC, true>(y, lane);
                    red_max[q4 * N + r0 + rr] = y[0];
                    if (half_any<L::H>(half, !ok || *abort_flag)) {
                        alive = false;
                        break;
                    }
                    bool moved = false;
                    if (t < NC) {
                        const int r = r0 + t;
                        const float best = fmaxf(fmaxf(red_max[r], red_max[N + r]),
                                                 fmaxf(red_max[2 * N + r], red_max[3 * N + r]));
                        const float old = first ? kUnset : s_m[r];
                        const float now = best > old + kSlack ? best : old;
                        s_alpha[r] = old == kUnset ? 1.f : fast_exp2(0.5f * (old - now));
                        s_m[r] = now;
                        moved = now != old && old != kUnset;
                    }
                    rescale = half_any<L::H>(half, moved);
                    unset = false;
#pragma unroll
                    for (int e = 0; e < NC; ++e) {
                        const float mx = s_m[r0 + e];
                        unset |= mx == kUnset;
                        nm[e] = mx == kUnset ? 0.f : kBoost - mx;
                        d[e] += nm[e];
                    }
                }
                // The PV product PB tiles back has read the weights' buffer (with two
                // buffers it had when this tile's scores came, which were issued behind
                // it); a rescale needs the last one in O as well.
                if (L::PB == 2 && g > 1) {
                    alive = __all_sync(kFull, await(&o_done[g & 1], ((g - 2) >> 1) & 1, abort_flag,
                                                    status));
                }
                if ((L::PB == 1 || rescale) && alive && g > 0) {
                    alive = __all_sync(kFull, await(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1,
                                                    abort_flag, status));
                    tc::tc_fence_after();
                }
                if (alive) {
                    if (rescale) {
#pragma unroll
                        for (int e = 0; e < NC; ++e) l[e] = l[e] * s_alpha[r0 + e] * s_alpha[r0 + e];
#pragma unroll 1
                        for (int z = 0; z < 3 * KS; ++z) {
                            uint32_t o[NC];
                            const uint32_t at =
                                tmem + L::kTmemO + z / 3 * L::PR + z % 3 * N + lanes + r0;
                            tmem_load<NC>(at, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < NC; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                                       (s_alpha[r0 + e] * s_alpha[r0 + e]));
                            tmem_store<NC>(at, o);
                        }
                        tc::tmem_st_wait();
                    }
                    // weights, two rows at a time: the thread's 16 bytes of key t, the two
                    // halves of 32 swapped in every other four keys; or byte t of row r of
                    // the K-major operand, 16-byte pieces swizzled by r % 8 (r0 and N are
                    // multiples of 8)
                    uint8_t *pw = s_p + g % L::PB * L::kPBytes +
                                  (L::kWide ? t * 32 + ((half ^ (t >> 2)) & 1) * 16
                                            : r0 * 128 + (t & 15));
                    uint32_t wide[3][NC / 4];
                    const __half2 eight = __floats2half2_rn(8.f, 8.f);
                    const uint64_t vs2 = pack2(vs, vs);
#pragma unroll
                    for (int e = 0; e < NC; e += 2) {
                        // the sum takes 2^d itself: a block of small (or zero) values has a
                        // small scale, and its keys' weights may vanish, not their share
                        const uint64_t x2 = pack2(fast_exp2(d[e]), fast_exp2(d[e + 1]));
                        unpack2(add2(pack2(l[e], l[e + 1]), x2), l[e], l[e + 1]);
                        float wa, wb;
                        unpack2(mul2(x2, vs2), wa, wb);
                        __half2 h = __floats2half2_rn(wa, wb);
                        uint8_t *pa = pw + ((((t >> 4) ^ e) & 7) << 4) + e * 128;
                        uint8_t *pb = pw + ((((t >> 4) ^ (e + 1)) & 7) << 4) + (e + 1) * 128;
#pragma unroll
                        for (int z = 0; z < 3; ++z) {
                            const uint32_t b = e5m2x2(h);
                            if constexpr (L::kWide) {
                                wide[z][e / 4] = e % 4 == 0 ? b : wide[z][e / 4] | b << 16;
                            } else {
                                pa[z * N * 128] = (uint8_t)b;
                                pb[z * N * 128] = (uint8_t)(b >> 8);
                            }
                            if (z < 2) h = __hmul2(__hsub2(h, e5m2x2_to_f16x2(b)), eight);
                        }
                    }
                    if constexpr (L::kWide) {
                        if constexpr (N == 8) {
                            *reinterpret_cast<uint4 *>(pw) =
                                make_uint4(wide[0][0], wide[0][1], wide[1][0], wide[1][1]);
                            *reinterpret_cast<uint2 *>(
                                reinterpret_cast<uintptr_t>(pw) ^ 16) =
                                make_uint2(wide[2][0], wide[2][1]);
                        } else {
#pragma unroll
                            for (int z = 0; z < 3; ++z)
                                *reinterpret_cast<uint4 *>(pw + z * kKeys * 32) =
                                    make_uint4(wide[z][0], wide[z][1], wide[z][2], wide[z][3]);
                        }
                    }
                    // A tile with rows outside the request's keys: their V bytes must not
                    // meet a zero weight (0 x NaN), so they are zeroed.  NaNs among the
                    // values of a key that only some queries see are taken out of the
                    // tile and put into those rows' weights instead.
                    bool nans = false;
                    if (edge && nq > 1) {
                        alive = __all_sync(kFull, await(&nan_full[si & 1], (si >> 1) & 1, abort_flag,
                                                        status));
                        nans = alive && sh->nans[si & 1];
                    }
                    if (t0 < lowest || t0 + kKeys > keys || nans) {
                        const uint32_t base = TS * (2 * g + (x + 1 < x1 ? 2 : 1));
                        // A wait for a phase by its parity means that phase only if the one
                        // before it is over: the stage may have been the last tile's V's.
                        if (g > 0 && !await(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag,
                                            status))
                            alive = false;
                        for (int z = 0; z < TS; ++z) {
                            const uint32_t c = base + z;
                            const int s = c % NS;
                            if (!await(&full[s], (c / NS) & 1, abort_flag, status)) {
                                alive = false;
                                break;
                            }
                            for (int y = half; !data && y < 2; y += L::H) {
                                uint4 *row = reinterpret_cast<uint4 *>(smem + s * kStage + y * kSlab +
                                                                       t * 128);
#pragma unroll
                                for (int q = 0; q < 8; ++q) row[q] = make_uint4(0, 0, 0, 0);
                            }
                        }
                        if (nans && alive && data &&
                            (pos > ctx || (p.window > 0 && pos < keys - p.window)) &&
                            remove_nans<D, NS>(p, smem, base, t, sg.b, sg.c, pos)) {
                            const uint32_t seen = seen_rows(pos);
#pragma unroll 1
                            for (int e = 0; e < NC; ++e)
                                if ((seen >> e) & 1u)
                                    pw[L::kWide ? e : ((((t >> 4) ^ e) & 7) << 4) + e * 128] = 0x7f;
                        }
                    }
                }
                alive = __all_sync(kFull, alive);
                tc::fence_proxy_async_smem();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&p_full[g & 1]);
                if (first && x + 1 < x1) have_next = it.next(p, nx);
            }
            // ------------------------------------------------ segment end
            // (a wait of one warp may have run out: all leave together)
            if (half_any<L::H>(half, !alive || *abort_flag)) {
                alive = false;
                break;
            }
            // While the last PV product runs: the rows' sums over the 128 keys.
            float y[NC];
#pragma unroll
            for (int e = 0; e < NC; ++e) y[e] = l[e] * kSum;
            const int rr = transpose_reduce<NC, false>(y, lane);
            red_max[q4 * N + r0 + rr] = y[0];
            half_any<L::H>(half, false);
            const size_t slot_row = ((size_t)blockIdx.x * 2 + (sg.opens ? 0 : 1)) * N + r0;
            if (t < NC) {
                const int r = r0 + t;
                float sum =
                    (red_max[r] + red_max[N + r]) + (red_max[2 * N + r] + red_max[3 * N + r]);
                // (more than 2^20 keys of next to nothing: the output is 0, not inf x 0)
                if (sum > 3e38f) sum = 3e38f;
                if (!whole) plan.part_ml[slot_row + t] = make_float2(s_m[r], sum * (1.f / kWeight));
                s_alpha[r] = 1.f / sum;
            }
            alive = __all_sync(kFull, await(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag,
                                            status));
            tc::tc_fence_after();
            if (half_any<L::H>(half, !alive || *abort_flag)) {
                alive = false;
                break;
            }
            // O of 8 rows and 128 d at a time: the pieces' sum (times kSum), then the output
            // row or the partial.  Rolled: this code runs once a segment, from an instruction
            // cache that holds the tile loop, and its fetches are its cost.
            const int parts = KS * ((min(rows_here - r0, NC) + 7) / 8);
            auto pieces = [&](int i, float (&o)[8]) {
                uint32_t o1[8], o2[8], o3[8];
                const uint32_t at = tmem + L::kTmemO + i % KS * L::PR + lanes + r0 + i / KS * 8;
                tc::tmem_ld8(at, o1);
                tc::tmem_ld8(at + N, o2);
                tc::tmem_ld8(at + 2 * N, o3);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = fmaf(fmaf(__uint_as_float(o3[e]), 0.125f, __uint_as_float(o2[e])), 0.125f,
                                __uint_as_float(o1[e])) * kSum;
            };
            if (whole) {
                // lanes 2i and 2i + 1 hold d and d + 1 of every row: one keeps the even
                // rows' pair, the other the odd rows', so stores are 4 bytes wide
                const bool odd = t & 1;
                const int base = out_row[0];   // the unit's first row here
#pragma unroll 1
                for (int i = 0; i < parts; ++i) {
                    float o[8];
                    pieces(i, o);
                    const int e0 = i / KS * 8;
                    const float4 fa = *reinterpret_cast<const float4 *>(s_alpha + r0 + e0);
                    const float4 fb = *reinterpret_cast<const float4 *>(s_alpha + r0 + e0 + 4);
                    const int4 ra = *reinterpret_cast<const int4 *>(out_row + e0);
                    const int4 rb = *reinterpret_cast<const int4 *>(out_row + e0 + 4);
                    const float f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
                    const int ro[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
                    uint16_t *out = p.out + (size_t)base * D + i % KS * 128 + (t & ~1);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float a = o[e] * f[e], b = o[e + 1] * f[e + 1];
                        const float got = __shfl_xor_sync(kFull, odd ? a : b, 1);
                        const __nv_bfloat162 h =
                            odd ? __floats2bfloat162_rn(got, b) : __floats2bfloat162_rn(a, got);
                        const int row = odd ? ro[e + 1] : ro[e];
                        if (row >= 0)
                            *reinterpret_cast<uint32_t *>(out + (long long)(row - base) * D) =
                                *reinterpret_cast<const uint32_t *>(&h);
                    }
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < parts; ++i) {
                    float o[8];
                    pieces(i, o);
                    float *po = plan.part_o + (slot_row + i / KS * 8) * D + i % KS * 128 + t;
#pragma unroll
                    for (int e = 0; e < 8; ++e) po[e * D] = o[e] * (1.f / kWeight);
                }
            }
            // all reads of the reduction area and of O come before the next segment's
            tc::tc_fence_before();
            half_any<L::H>(half, false);
            if (lane == 0) tc::mbar_arrive(&q_free[si & 1]);
            have = have_next;
            sg = nx;
            ++si;
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tc::tmem_dealloc(sh->tmem, L::kTmem);
    }
}

// Merge of the split units: out = sum_q 2^(m_q - M) O_q / sum_q 2^(m_q - M) l_q
// over the pieces q, M their largest maximum (a piece whose l is 0 saw no key of
// the row).  2^(m_q - M) may underflow where its product with l_q is the larger part
// of the sum (see the sum's range above): it is two factors, applied in turn.  A CTA takes `rows` rows of one unit and row group; a row has D / 4
// threads of 16 bytes each, `teams` times over: the teams take the pieces in
// turn, so that a unit cut into many pieces has many loads in flight, F a thread.
// F = 8 and teams for more than 8 pieces a unit (one request of 6005 keys, 47 pieces:
// 4.4 us); F = 3 of 32 bytes else, with two CTAs an SM (64 x 4, at most a few pieces:
// 5 us, about 60 MB read and written).
constexpr int kMergeThreads = 512, kMergeRows = 8;

template <int D, int N, int F>
__global__ void __launch_bounds__(kMergeThreads, F > 4 ? 1 : 2) paged_fp8_merge_kernel(
    const __grid_constant__ PagedFp8Params p, const Plan plan, int rows, int teams) {
    constexpr int V = F > 4 ? 1 : 2, T = D / 4 / V;   // 16-byte vectors a thread
    wait_for_prior_launch();
    let_next_launch_start();
    const int u = blockIdx.x;
    const int rg = u % plan.groups, bc = u / plan.groups;
    const int b = bc / p.kv_heads, c = bc % p.kv_heads;
    const Request rq = load_request(p, b);
    const int2 e = plan.first[u];
    const int np = plan.last[u] - e.x + 1;
    if (!request_ok(p, rq) || rq.n == 0) return;
    if (e.y < 0) return;   // whole: written already
    // entries that the attention grid did not write this time (it gave up before)
    if (e.x < 0 || np < 2 || np > kMaxPieces || e.x > plan.ranges - np || e.y > 1) {
        if (threadIdx.x == 0) set_status(p.dev_status, CARAT_DEV_TIMEOUT);
        return;
    }
    const int d = threadIdx.x % T, rt = threadIdx.x / T;
    const int team = rt / rows, mine = rt % rows;
    const int r = blockIdx.y * rows + mine, ur = rg * N + r;
    const bool valid = r < N && ur < p.group * rq.n;
    auto piece = [&](int q) -> size_t {
        return ((size_t)((e.x + q) * plan.groups + rg) * 2 + (q == 0 ? e.y : 0)) * N + r;
    };
    __shared__ float s_w[kMergeRows][kMaxPieces];
    __shared__ float4 s_o[F > 4 ? kMergeThreads : 1];
    const int lane = threadIdx.x % 32;
    // the first pieces' values on their way before the weights are formed
    float4 v[F][V];
    auto load = [&](int q0) {
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int q = q0 + i * teams;
            if (!valid || q >= np) continue;
            const float4 *o = reinterpret_cast<const float4 *>(plan.part_o + piece(q) * D) + d;
#pragma unroll
            for (int z = 0; z < V; ++z) v[i][z] = o[z * T];
        }
    };
    load(team);
    if (valid && team == 0 && d < 32) {
        float M = kUnset, sum = 0.f;
        if constexpr (F > 4) {   // many pieces: all of them in registers at once
            constexpr int G = kMaxPieces / 32;
            float2 ml[G];
#pragma unroll
            for (int i = 0; i < G; ++i)
                ml[i] = lane + 32 * i < np ? plan.part_ml[piece(lane + 32 * i)]
                                           : make_float2(kUnset, 0.f);
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (ml[i].y != 0.f) M = fmaxf(M, ml[i].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
#pragma unroll
            for (int i = 0; i < G; ++i) {
                ml[i].x = ml[i].y != 0.f ? fast_exp2(0.5f * (ml[i].x - M)) : 0.f;
                sum = fmaf(ml[i].x, ml[i].x * ml[i].y, sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            const float inv = 1.f / sum;
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (lane + 32 * i < np) s_w[mine][lane + 32 * i] = ml[i].x * inv * ml[i].x;
        } else {                 // a few
            for (int q = lane; q < np; q += 32) {
                const float2 ml = plan.part_ml[piece(q)];
                if (ml.y != 0.f) M = fmaxf(M, ml.x);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
            for (int q = lane; q < np; q += 32) {
                const float2 ml = plan.part_ml[piece(q)];
                const float w = ml.y != 0.f ? fast_exp2(0.5f * (ml.x - M)) : 0.f;
                s_w[mine][q] = w;
                sum = fmaf(w, w * ml.y, sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            const float inv = 1.f / sum;
            for (int q = lane; q < np; q += 32) s_w[mine][q] *= inv * s_w[mine][q];
        }
    }
    __syncthreads();
    float4 acc[V] = {};
#pragma unroll 1
    for (int q0 = team; q0 < np; q0 += F * teams) {
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int q = q0 + i * teams;
            if (!valid || q >= np) continue;
            const float w = s_w[mine][q];
            if (w == 0.f) continue;
#pragma unroll
            for (int z = 0; z < V; ++z) {
                acc[z].x = fmaf(v[i][z].x, w, acc[z].x);
                acc[z].y = fmaf(v[i][z].y, w, acc[z].y);
                acc[z].z = fmaf(v[i][z].z, w, acc[z].z);
                acc[z].w = fmaf(v[i][z].w, w, acc[z].w);
            }
        }
        load(q0 + F * teams);
    }
    if constexpr (F > 4) {
        s_o[threadIdx.x] = acc[0];
        __syncthreads();
        if (team > 0) return;
        for (int i = 1; i < teams; ++i) {
            const float4 w = s_o[(i * rows + mine) * T + d];
            acc[0].x += w.x, acc[0].y += w.y, acc[0].z += w.z, acc[0].w += w.w;
        }
    }
    if (!valid) return;
    const int j = ur / p.group;
    const size_t row = ((size_t)b * p.k + j) * p.q_heads + (size_t)c * p.group + ur - j * p.group;
#pragma unroll
    for (int z = 0; z < V; ++z) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[z].x, acc[z].y);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[z].z, acc[z].w);
        reinterpret_cast<uint2 *>(p.out + row * D)[d + z * T] =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                       *reinterpret_cast<const uint32_t *>(&hi));
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Rows of a tile: 8, 16, or groups of 32.
int tile_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

struct Sizes {
    int n, groups, grid;
    size_t ml, o, units, last, total;
};

Sizes sizes_of(int batch, int k, int q_heads, int kv_heads, int head_dim) {
    Sizes z{};
    const int rows = q_heads / kv_heads * k;
    z.n = tile_rows(rows);
    z.groups = (rows + z.n - 1) / z.n;
    const int sms = device_sm_count();
    const int slots_sm = head_dim == 256 && z.n <= 16 ? Lay<256, 16>::OCC : 1;
    const int ranges = std::min(slots_sm * sms / z.groups, kMaxPieces);
    z.grid = (ranges < 1 ? 1 : ranges) * z.groups;
    const size_t slots = (size_t)z.grid * 2 * z.n;
    z.ml = align256(slots * sizeof(float2));
    z.o = align256(slots * (size_t)head_dim * sizeof(float));
    const size_t count = (size_t)batch * kv_heads * z.groups;
    z.units = align256(count * sizeof(int2));
    z.last = align256(count * sizeof(int));
    // Image<head_dim, n>
    z.total = z.ml + z.o + z.units + z.last + align256(count * (2 * z.n * (head_dim + 4)));
    return z;
}

template <int D, int N>
cudaError_t launch(const PagedFp8Params &p, const Sizes &z, cudaStream_t stream) {
    using L = Lay<D, N>;
    Plan plan{};
    plan.groups = z.groups;
    plan.ranges = z.grid / z.groups;
    char *w = static_cast<char *>(p.workspace);
    plan.part_ml = reinterpret_cast<float2 *>(w);
    plan.part_o = reinterpret_cast<float *>(w + z.ml);
    plan.first = reinterpret_cast<int2 *>(w + z.ml + z.o);
    plan.last = reinterpret_cast<int *>(w + z.ml + z.o + z.units);
    plan.images = reinterpret_cast<uint8_t *>(w + z.ml + z.o + z.units + z.last);
    // (128 d, rows, 128-d block, head); a stage is 128 rows of two blocks
    CUtensorMap map_k{}, map_v{};
    const uint64_t row = (uint64_t)p.kv_heads * D;
    const uint64_t dims[4] = {128, (uint64_t)p.num_pages * p.page_rows, D / 128,
                              (uint64_t)p.kv_heads};
    const uint64_t strides[3] = {row, 128, D};
    const uint32_t box[4] = {128, kKeys, 2, 1};
    if (!make_u8_tensor_map(&map_k, p.k_pages, 4, dims, strides, box, true) ||
        !make_u8_tensor_map(&map_v, p.v_pages, 4, dims, strides, box, true))
        return cudaErrorInvalidValue;
    auto kernel = paged_fp8_kernel<D, N>;
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(1, std::memory_order_release);
    }
    // The attention may start while the split launch runs, and the merge while the
    // attention drains; each waits where it needs the other's results.
    const int units = p.batch * p.kv_heads * z.groups;
    e = launch_dependent(paged_fp8_split_kernel<D, N>, dim3(units), dim3(32 * N), 0, stream, p, plan);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, dim3(z.grid), dim3(L::kThreads), L::kAlloc, stream, p, plan, map_k,
                         map_v);
    if (e != cudaSuccess) return e;
    // A unit is cut into about ranges / units + 1 pieces.  One long unit among short
    // ones, cut into many more, is walked by the threads of a few: its lengths are on the
    // device (what that costs: see the head of this file).
    const int held = std::min(N, p.group * p.k);
    const int pieces = plan.ranges / (p.batch * p.kv_heads) + 1;
    const bool many = pieces > 8;
    const int row_threads = many ? D / 4 : D / 8, most = kMergeThreads / row_threads;
    int teams = 1, rows = 1;
    while (many && teams < most && pieces > 8 * teams) teams *= 2;
    while (rows < kMergeRows && rows * teams < most && rows < held) rows *= 2;
    auto merge = many ? paged_fp8_merge_kernel<D, N, 8> : paged_fp8_merge_kernel<D, N, 3>;
    return launch_dependent(merge, dim3(units, (held + rows - 1) / rows),
                            dim3(row_threads * rows * teams), 0, stream, p, plan, rows, teams);
}

}  // namespace

bool paged_fp8_supported(int head_dim) { return head_dim == 256 || head_dim == 512; }

size_t paged_fp8_workspace(int batch, int proposal_count, int q_heads, int kv_heads,
                           int head_dim) {
    return batch > 0 ? sizes_of(batch, proposal_count, q_heads, kv_heads, head_dim).total : 0;
}

cudaError_t launch_paged_fp8_attention(const PagedFp8Params &p, cudaStream_t stream) {
    const Sizes z = sizes_of(p.batch, p.k, p.q_heads, p.kv_heads, p.head_dim);
    if (p.head_dim == 256)
        return z.n == 8    ? launch<256, 8>(p, z, stream)
               : z.n == 16 ? launch<256, 16>(p, z, stream)
                           : launch<256, 32>(p, z, stream);
    return z.n == 8    ? launch<512, 8>(p, z, stream)
           : z.n == 16 ? launch<512, 16>(p, z, stream)
                       : launch<512, 32>(p, z, stream);
}

}  // namespace carat
