// paged_chunk.cu -- attention of a chunk of new tokens over bf16 pages.
//
// Query j of request b sits at position p = context_lengths[b] + j and sees key t when
//   t <= p  and  (window == 0  or  t > p - window  or  t < sinks);
//   out = sum_t softmax_t(scale q . k_t) v_t over the keys it sees.
//
// Rows.  The query heads that share a KV head and the chunk's tokens form rows r = j*g + h'
// (g = q_heads / kv_heads); a CTA holds the 128 / g tokens whose rows fill 128, a pair of
// CTAs (a cluster of two SMs) twice as many, and each key tile of 128 keys is loaded once
// for the pair, half by each:
//     S [256 rows x 128 keys] = Q . K_tile^T      A: own 128 rows, B: 64 keys a CTA
//     O [256 rows x 256 d]   += P . V_tile        A: own rows of P, B: 128 d a CTA
// tcgen05.mma cta_group::2, bf16 operands, fp32 accumulators.  Tensor memory of a CTA: O 256
// columns, two S tiles of 128; P (bf16) takes the place of the S tile it comes from and is
// read from there.  At head_dim 512 O of 128 rows would fill all 512 columns, so a pair
// takes one half of the value dimensions and the scores are computed for each half again
// (1.5 times the operations).
//
// What bounds it: the tensor pipe.  A pair reads K and V tiles at 32 bytes a cycle and SM
// from L2, against 64 without pairs, which L2 could not give.
//
// Softmax.  One thread a row, 128 keys of a tile in registers.  The running maximum is
// replaced only when a tile exceeds it by more than 8 (log2 units), so O is rarely read
// back and rescaled; P <= 2^8.  P is rounded to bf16 (the tensor core's operand, with V
// bf16; 2^-8 of each weight) and the rounded weights are summed, so numerator and
// denominator see the same ones.
//
// Keys.  An item (request, KV head, row tile, value half, split) walks the tiles that hold
// a key some row of the pair sees: those of the sinks, then from the first row's window to
// the last row's position.  A tile some row sees only in part is masked by position.  Its
// V rows could carry what no row may see into O through 0 x infinity: the softmax threads
// look through such a tile's V for values that are not finite and zero those rows, and
// rows behind the last key, before the product; a row that sees such a key is written as
// NaN.
//
// Few items (fewer than pairs of SMs): the key tiles of an item are split over CTA pairs,
// each writes (max, sum, unnormalised O), and a second launch merges them.
//
// Warp roles (256 threads): warp 0 TMA producer (each CTA its own halves, counted on the
// leader's barriers), warp 1 of the leader issues the products, warps 4-7 softmax, rescale
// and output.  Every wait is bounded: on a timeout CARAT_DEV_TIMEOUT is set and the CTA
// stops, waits for its own copies and products, and returns.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

#include <cuda_bf16.h>

#include "carat_internal.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace carat {
namespace {

constexpr int kKeys = 128;              // keys of a tile
constexpr int kRows = 128;              // rows of a CTA
constexpr int kDV = 256;                // value dimensions of an item
constexpr int kStage = 32768;           // K: 64 keys x 256 d, or V: 128 keys x 128 d
constexpr int kThreads = 256;
constexpr int kMasked = 8;              // masked tiles of an item: 3 + 3 + 1 at most
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kSlack = 8.0f;          // log2 units

template <int D>
struct Lay {
    static constexpr int KST = D / 256;                 // stages of a K tile
    static constexpr int NS = D == 256 ? 5 : 3;         // stage ring
    static constexpr int kSlab = kRows * 128;           // 64 d of Q
    static constexpr int kOffQ = NS * kStage;
    static constexpr int kOffMisc = kOffQ + D / 64 * kSlab;
    static constexpr int kBytes = kOffMisc + 1024;
    static constexpr int kAlloc = kBytes + 1024;        // base alignment
    static_assert(kAlloc <= 232448, "more dynamic shared memory than one CTA may use");
};

template <int NS>
struct Shared {
    uint64_t full[NS];      // leader: a stage's bytes of both CTAs have landed
    uint64_t empty[NS];     // both: the products that read the stage are done
    uint64_t q_full;        // leader
    uint64_t s_full[2];     // both: a tile's scores are in tensor memory
    uint64_t p_full[2];     // leader: its weights are, and V is looked through
    uint64_t pv_done;       // both: a tile's value product is done
    uint64_t v_ready;       // both: a masked tile's V has landed
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int poison;             // some masked tile held a value that is not finite
    int tile_base[kMasked];
    uint32_t bad[kMasked][2][4];   // such keys of masked tile i, by CTA of the pair
};

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

struct Plan {
    int tokens;      // of a CTA
    int tiles;       // row tiles (of a pair) of a request's chunk
    int halves;      // value halves
    int splits;
    float2 *part_ml; // [B k Hq][splits]
    float *part_o;   // [B k Hq][splits][D]
};

// Key tiles of the rows at positions [lo, hi]: the sinks', then the window's.
struct Keys {
    long long lo, hi;
    long long first;
    int sink_tiles, count;

    __device__ __forceinline__ Keys(const PagedChunkParams &p, long long lo_, long long hi_)
        : lo(lo_), hi(hi_) {
        first = p.window > 0 && lo - p.window + 1 > 0 ? (lo - p.window + 1) / kKeys : 0;
        const long long s = p.window > 0 ? ((long long)p.sinks + kKeys - 1) / kKeys : 0;
        sink_tiles = (int)(s < first ? s : first);
        count = sink_tiles + (int)(hi / kKeys - first) + 1;
    }
    __device__ __forceinline__ long long base(int x) const {
        return (x < sink_tiles ? x : first + x - sink_tiles) * kKeys;
    }
    // whether some row sees some key of the tile at t0 and not another
    __device__ __forceinline__ bool masked(const PagedChunkParams &p, long long t0) const {
        if (t0 + kKeys - 1 > lo) return true;
        return p.window > 0 && t0 <= hi - p.window && t0 + kKeys > p.sinks;
    }
};

// Pieces of `count` tiles: split s takes [count s / splits, count (s + 1) / splits).
__device__ __forceinline__ int split_at(int count, int s, int splits) {
    return (int)((long long)count * s / splits);
}

// Bounded wait; false on a timeout or when another role of this CTA gave up.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity,
                                              volatile int *abort_flag, int *dev_status) {
    if (tc::mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    for (uint32_t round = 1;; ++round) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (tc::mbar_try_wait_cluster(bar, parity)) return true;
        if (*abort_flag) return false;
        if (tc::wait_expired(t0, round, 2000000000ull)) {
            *abort_flag = 1;
            set_status(dev_status, CARAT_DEV_TIMEOUT);
            return false;
        }
    }
}

// The same for a whole warp, which goes on or stops as one.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity,
                                          volatile int *abort_flag, int *dev_status) {
    return __all_sync(kFull, wait_or_abort(bar, parity, abort_flag, dev_status)) != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// An offset into a tile, held within [-1, kKeys].
__device__ __forceinline__ int within(long long x) {
    return (int)(x < -1 ? -1 : x > kKeys ? kKeys : x);
}

__device__ __forceinline__ void softmax_barrier() {
    asm volatile("bar.sync 1, 128;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    paged_chunk_kernel(const __grid_constant__ PagedChunkParams p, const Plan plan,
                       const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v) {
    using L = Lay<D>;
    constexpr int NS = L::NS, KST = L::KST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto *sh = reinterpret_cast<Shared<NS> *>(smem + L::kOffMisc);
    static_assert(sizeof(Shared<NS>) <= 1024, "misc area");
    uint8_t *s_q = smem + L::kOffQ;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)tc::cluster_ctarank();

    wait_for_prior_launch();
    let_next_launch_start();

    // The item: later row tiles (longer under a causal mask) come first.
    int idx = blockIdx.x / 2;
    const int split = idx % plan.splits;
    idx /= plan.splits;
    const int vh = idx % plan.halves;
    idx /= plan.halves;
    const int c = idx % p.kv_heads;
    idx /= p.kv_heads;
    const int b = idx % p.batch;
    const int tile = plan.tiles - 1 - idx / p.batch;
    const Request rq = load_request(p, b);
    const int j0 = tile * 2 * plan.tokens;          // the pair's first token
    const int mine = j0 + rank * plan.tokens;       // this CTA's
    if (!request_ok(p, rq)) {
        if (split == 0) {
            for (int i = threadIdx.x; i < plan.tokens * p.group * (kDV / 8); i += kThreads) {
                const int r = i / (kDV / 8), j = mine + r / p.group;
                if (j < p.k)
                    *reinterpret_cast<uint4 *>(
                        p.out + (((size_t)b * p.k + j) * p.q_heads + c * p.group + r % p.group) * D +
                        vh * kDV + i % (kDV / 8) * 8) =
                        make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            }
            if (threadIdx.x == 0) set_status(p.dev_status, CARAT_DEV_BAD_CONTEXT);
        }
        return;
    }
    if (j0 >= rq.n) return;
    const int jend = min(j0 + 2 * plan.tokens, rq.n);
    const Keys keys(p, rq.ctx + j0, rq.ctx + jend - 1);
    const int x0 = split_at(keys.count, split, plan.splits);
    const int n = split_at(keys.count, split + 1, plan.splits) - x0;
    if (n == 0) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&sh->full[i], 1);
            tc::mbar_init(&sh->empty[i], 1);
        }
        tc::mbar_init(&sh->q_full, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh->s_full[i], 1);
            tc::mbar_init(&sh->p_full[i], 8);
        }
        tc::mbar_init(&sh->pv_done, 1);
        tc::mbar_init(&sh->v_ready, 1);
        tc::mbar_init(&sh->drain, 1);
        tc::fence_mbar_init();
        sh->abort_flag = 0;
        sh->poison = 0;
    }
    if (threadIdx.x < kMasked * 8) (&sh->bad[0][0][0])[threadIdx.x] = 0;
    if (warp == 1) {
        tc::tmem_alloc_pair(&sh->tmem, 512);
        tc::tmem_relinquish_pair();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();
    tc::tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const uint32_t t_o = tmem, t_s = tmem + kDV;
    volatile int *abort_flag = &sh->abort_flag;

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        uint32_t cnt = 0;
        bool alive = true;
        const uint32_t q_bytes = plan.tokens * p.group * 128;
        if (lane == 0) {
            if (rank == 0) tc::mbar_arrive_expect_tx(&sh->q_full, 2 * (D / 64) * q_bytes);
            const uint32_t bar = tc::map_to_rank(&sh->q_full, 0);
            for (int i = 0; i < D / 64; ++i)
                tc::tma_load_4d_pair(s_q + i * L::kSlab, &map_q, i * 64, c * p.group, mine, b, bar);
        }
        int row_held = 0;   // lane l: pool row of tile 32 * (x / 32) + l
        auto row_of = [&](int x) -> int {
            return __shfl_sync(kFull, row_held, x & 31);
        };
        auto fetch = [&](int x) {   // rows of the 32 tiles from x on
            const int mine_x = x + lane;
            if (mine_x < n) {
                const long long t = keys.base(x0 + mine_x);
                const int page = p.page_table[(size_t)b * p.max_pages + (int)(t / p.page_rows)];
                if (page < 0 || page >= p.num_pages) {
                    set_status(p.dev_status, CARAT_DEV_BAD_CACHE_ID);
                    row_held = -1;
                } else {
                    row_held = page * p.page_rows + (int)(t % p.page_rows);
                }
            }
        };
        auto load = [&](bool is_v, int row, int part) {
            const int s = cnt % NS;
            if (cnt >= NS && alive)
                alive = warp_wait(&sh->empty[s], ((cnt / NS) & 1) ^ 1, abort_flag, p.dev_status);
            if (!alive) return;
            if (lane == 0) {
                if (rank == 0) tc::mbar_arrive_expect_tx(&sh->full[s], 2 * kStage);
                const uint32_t bar = tc::map_to_rank(&sh->full[s], 0);
                // a page outside the pool: rows behind the tensor's end read as zeros
                const int at = row < 0 ? p.num_pages * p.page_rows : row + (is_v ? 0 : rank * 64);
                if (is_v)
                    tc::tma_load_4d_pair(smem + s * kStage, &map_v, 0, at, vh * 4 + rank * 2, c, bar);
                else
                    tc::tma_load_4d_pair(smem + s * kStage, &map_k, 0, at, part * 4, c, bar);
            }
            ++cnt;
        };
        int prev = 0;
        for (int x = 0; x <= n && alive; ++x) {
            int row = 0;
            if (x < n) {
                if ((x & 31) == 0) fetch(x);
                row = row_of(x);
                for (int k = 0; k < KST; ++k) load(false, row, k);
            }
            if (x > 0) load(true, prev, 0);
            prev = row;
        }
        if (!alive && rank == 0) {
            // let what both CTAs' copies still carry land before anyone leaves
            for (uint32_t i = cnt > NS ? cnt - NS : 0; i < cnt; ++i)
                tc::mbar_wait(&sh->full[i % NS], (i / NS) & 1);
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------------- products
        const bool negative = p.scale_log2 < 0.f;
        const uint32_t id_qk = tc::idesc_bf16_f32(256, kKeys, false, false) |
                               (negative ? 1u << 13 : 0u);   // negates A
        constexpr uint32_t id_pv = tc::idesc_bf16_f32(256, kDV, false, true);
        const uint32_t q_addr = tc::smem_u32(s_q), st_addr = tc::smem_u32(smem);
        uint32_t cnt = 0;
        bool alive = warp_wait(&sh->q_full, 0, abort_flag, p.dev_status);
        for (int x = 0; x <= n && alive; ++x) {
            if (x < n) {
                for (int k = 0; k < KST && alive; ++k, ++cnt) {
                    const int s = cnt % NS;
                    alive = warp_wait(&sh->full[s], (cnt / NS) & 1, abort_flag, p.dev_status);
                    if (!alive) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t off = (i & 3) * 32;
                        tc::mma_bf16_ss_pair(
                            t_s + (x & 1) * kKeys,
                            tc::sdesc_sw128(q_addr + (k * 4 + i / 4) * L::kSlab + off, 16, 1024),
                            tc::sdesc_sw128(st_addr + s * kStage + i / 4 * 8192 + off, 16, 1024),
                            id_qk, k > 0 || i > 0);
                    }
                    tc::mma_commit_pair(&sh->empty[s]);
                }
                if (!alive) break;
                tc::mma_commit_pair(&sh->s_full[x & 1]);
            }
            if (x == 0) continue;
            const int y = x - 1, s = cnt % NS;
            alive = warp_wait(&sh->full[s], (cnt / NS) & 1, abort_flag, p.dev_status);
            if (!alive) break;
            if (keys.masked(p, keys.base(x0 + y)) && lane == 0) {
                tc::mbar_arrive_cluster(tc::map_to_rank(&sh->v_ready, 0));
                tc::mbar_arrive_cluster(tc::map_to_rank(&sh->v_ready, 1));
            }
            __syncwarp();
            alive = warp_wait(&sh->p_full[y & 1], (y / 2) & 1, abort_flag, p.dev_status);
            if (!alive) break;
            tc::tc_fence_after();
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
                tc::mma_bf16_ts_pair(t_o, t_s + (y & 1) * kKeys + i * 8,
                                     tc::sdesc_sw128(st_addr + s * kStage + i * 2048, 16384, 1024),
                                     id_pv, y > 0 || i > 0);
            tc::mma_commit_pair(&sh->empty[s]);
            tc::mma_commit_pair(&sh->pv_done);
            ++cnt;
        }
        if (!alive) {
            tc::mma_commit_pair(&sh->drain);
            tc::mbar_wait(&sh->drain, 0);
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax
        const int row = threadIdx.x - 128;              // TMEM lane
        const uint32_t quad = (uint32_t)(warp - 4) << 21;
        const int j = mine + row / p.group, h = c * p.group + row % p.group;
        const bool valid = row < plan.tokens * p.group && j < rq.n;
        const long long pos = rq.ctx + j;
        // the sign of the scale is in the product's descriptor; 0 would turn -inf into NaN
        const float scale = fmaxf(fabsf(p.scale_log2), FLT_MIN);
        float m = -INFINITY, l = 0.f;
        int masked_tiles = 0;
        bool alive = true;
        for (int x = 0; x < n && alive; ++x) {
            alive = warp_wait(&sh->s_full[x & 1], (x / 2) & 1, abort_flag, p.dev_status);
            if (!alive) break;
            tc::tc_fence_after();
            const uint32_t t_x = t_s + (x & 1) * kKeys + quad;
            uint32_t s[kKeys];
#pragma unroll
            for (int i = 0; i < kKeys; i += 32) tc::tmem_ld32(t_x + i, s + i);
            tc::tmem_ld_wait();
            const long long t0 = keys.base(x0 + x);
            const bool masked = keys.masked(p, t0);
            if (masked) {
                const int hi = within(pos - t0);
                const int lo = p.window > 0 ? within(pos - p.window + 1 - t0) : -1;
                const int sk = within(p.sinks - t0);
#pragma unroll
                for (int i = 0; i < kKeys; ++i)
                    if (i > hi || (i < lo && i >= sk)) s[i] = 0xff800000u;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kKeys; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(s[i]));
            const float tm = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
            const bool grow = tm > m + kSlack || (m == -INFINITY && tm > m);
            if (__any_sync(kFull, grow)) {
                const float m_new = grow ? tm : m;
                const float f = m == m_new ? 1.f : fast_exp2(m - m_new);
                m = m_new;
                l *= f;
                if (x > 0) {
                    alive = warp_wait(&sh->pv_done, (x - 1) & 1, abort_flag, p.dev_status);
                    if (!alive) break;
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < kDV; i += 32) {
                        uint32_t o[32];
                        tc::tmem_ld32(t_o + quad + i, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st32(t_o + quad + i, o);
                    }
                    tc::tmem_st_wait();
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kKeys; i += 2) {
                const float a = fast_exp2(fmaf(__uint_as_float(s[i]), scale, -ref));
                const float d = fast_exp2(fmaf(__uint_as_float(s[i + 1]), scale, -ref));
                const uint32_t w = pack_bf16(a, d);
                s[i / 2] = w;
                sum[i / 2 & 3] += bf16lo(w) + bf16hi(w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc::tmem_st32(t_x, s);
            tc::tmem_st32(t_x + 32, s + 32);
            tc::tmem_st_wait();
            if (masked) {
                // V rows that not every row of the pair sees: nothing that is not finite
                // may meet a weight of 0.  Thread t looks through key t.
                alive = warp_wait(&sh->v_ready, masked_tiles & 1, abort_flag, p.dev_status);
                if (!alive) break;
                // stages in order: K(0), K(1) V(0), K(2) V(1), ..., V(n - 1)
                const int stage = ((x + 1 < n ? x + 2 : n) * KST + x) % NS;
                uint8_t *v_row = smem + stage * kStage + row * 128;
                bool bad = false;
                const bool stale = t0 + row > keys.hi;
                if (!stale) {
                    __nv_bfloat162 acc = __float2bfloat162_rn(0.f);
                    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            v_row + (i >> 3) * 16384 + ((i + row) & 7) * 16);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x), zero, acc);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y), zero, acc);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.z), zero, acc);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.w), zero, acc);
                    }
                    bad = __hisnan(acc.x) || __hisnan(acc.y);
                }
                if (bad || stale) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        *reinterpret_cast<uint4 *>(v_row + (i >> 3) * 16384 + (i & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    tc::fence_proxy_async_smem();
                }
                const uint32_t mask = __ballot_sync(kFull, bad);
                if (lane == 0) {
                    sh->tile_base[masked_tiles] = (int)t0;
                    if (mask) {
                        for (int r = 0; r < 2; ++r) {
                            tc::st_cluster_u32(tc::map_to_rank(&sh->bad[masked_tiles][rank][warp - 4], r),
                                               mask);
                            tc::st_cluster_u32(tc::map_to_rank(&sh->poison, r), 1);
                        }
                    }
                }
                ++masked_tiles;
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(tc::map_to_rank(&sh->p_full[x & 1], 0));
        }
        // The last scores say that the product two tiles before is done, no more: a wait for
        // the last product alone could pass on that one's phase, which has its parity.
        if (alive && n > 1) alive = warp_wait(&sh->pv_done, n & 1, abort_flag, p.dev_status);
        if (alive) alive = warp_wait(&sh->pv_done, (n - 1) & 1, abort_flag, p.dev_status);
        softmax_barrier();
        if (alive && !*abort_flag) {
            tc::tc_fence_after();
            bool poisoned = false;
            if (*(volatile int *)&sh->poison) {
                for (int i = 0; i < masked_tiles; ++i)
                    for (int w = 0; w < 4; ++w)
                        for (uint32_t bits = sh->bad[i][0][w] | sh->bad[i][1][w]; bits; bits &= bits - 1) {
                            const long long t = (long long)sh->tile_base[i] + w * 32 + __ffs(bits) - 1;
                            poisoned |= t <= pos && (p.window == 0 || t > pos - p.window || t < p.sinks);
                        }
            }
            // 128 bytes of each of the warp's 32 rows at a time through shared memory (Q's,
            // which no product reads any more), so that a row leaves as whole lines
            uint8_t *stage = s_q + (warp - 4) * 4096;
            const bool partial = plan.splits > 1;
            const float f = poisoned ? NAN : partial ? 1.f : 1.f / l;
            const size_t out_row = ((size_t)b * p.k + j) * p.q_heads + h;
            if (partial && valid && vh == 0)
                plan.part_ml[out_row * plan.splits + split] = make_float2(m, l);
#pragma unroll 1
            for (int i = 0; i < kDV; i += 64) {
                uint32_t o[64];
                tc::tmem_ld32(t_o + quad + i, o);
                tc::tmem_ld32(t_o + quad + i + 32, o + 32);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 64; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!partial && half) break;
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint4 v;
                        if (partial) {
                            const uint32_t *from = o + half * 32 + e * 4;
                            v = make_uint4(from[0], from[1], from[2], from[3]);
                        } else {
                            uint32_t w[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                w[z] = pack_bf16(__uint_as_float(o[e * 8 + 2 * z]),
                                                 __uint_as_float(o[e * 8 + 2 * z + 1]));
                            v = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((e ^ lane) & 7) * 16) = v;
                    }
                    __syncwarp();
                    for (int r8 = 0; r8 < 32; r8 += 4) {
                        const int r = r8 + lane / 8, e = lane % 8;
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            stage + r * 128 + ((e ^ r) & 7) * 16);
                        const int rr = (warp - 4) * 32 + r;
                        const int jj = mine + rr / p.group;
                        if (rr >= plan.tokens * p.group || jj >= rq.n) continue;
                        const size_t at =
                            ((size_t)b * p.k + jj) * p.q_heads + c * p.group + rr % p.group;
                        if (partial)
                            *reinterpret_cast<uint4 *>(plan.part_o + (at * plan.splits + split) * D +
                                                       vh * kDV + i + half * 32 + e * 4) = v;
                        else
                            *reinterpret_cast<uint4 *>(p.out + at * D + vh * kDV + i + e * 8) = v;
                    }
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_arrive();
    tc::cluster_wait();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, 512);
    }
}

// Merges the pieces of split items: one CTA a row of the output.
template <int D>
__global__ void __launch_bounds__(D / 4) paged_chunk_merge_kernel(
    const __grid_constant__ PagedChunkParams p, const Plan plan) {
    wait_for_prior_launch();
    let_next_launch_start();
    const int j = blockIdx.x / p.q_heads % p.k, b = blockIdx.x / p.q_heads / p.k;
    const Request rq = load_request(p, b);
    if (!request_ok(p, rq) || j >= rq.n) return;
    const int j0 = j / (2 * plan.tokens) * 2 * plan.tokens;
    const Keys keys(p, rq.ctx + j0, rq.ctx + min(j0 + 2 * plan.tokens, rq.n) - 1);
    const size_t at = blockIdx.x;
    float top = -INFINITY;
    for (int s = 0; s < plan.splits; ++s)
        if (split_at(keys.count, s, plan.splits) < split_at(keys.count, s + 1, plan.splits))
            top = fmaxf(top, plan.part_ml[at * plan.splits + s].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int s = 0; s < plan.splits; ++s) {
        if (split_at(keys.count, s, plan.splits) == split_at(keys.count, s + 1, plan.splits))
            continue;
        const float2 ml = plan.part_ml[at * plan.splits + s];
        const float w = fast_exp2(ml.x - ref);
        const float4 v =
            reinterpret_cast<const float4 *>(plan.part_o + (at * plan.splits + s) * D)[threadIdx.x];
        sum = fmaf(w, ml.y, sum);
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    }
    const float f = 1.f / sum;
    reinterpret_cast<uint2 *>(p.out + at * D)[threadIdx.x] =
        make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Sizes {
    Plan plan;
    long long items;    // CTA pairs
    size_t ml, total;
};

Sizes sizes_of(int batch, int k, int q_heads, int kv_heads, int head_dim) {
    Sizes z{};
    const int group = q_heads / kv_heads;
    z.plan.tokens = kRows / group;
    z.plan.tiles = (k + 2 * z.plan.tokens - 1) / (2 * z.plan.tokens);
    z.plan.halves = head_dim / kDV;
    z.items = (long long)batch * kv_heads * z.plan.tiles * z.plan.halves;
    const int pairs = device_sm_count() / 2;
    z.plan.splits = z.items > 0 && z.items <= pairs / 2 ? (int)(pairs / z.items) : 1;
    if (z.plan.splits > 1) {
        const size_t rows = (size_t)batch * k * q_heads * z.plan.splits;
        z.ml = align256(rows * sizeof(float2));
        z.total = z.ml + align256(rows * head_dim * sizeof(float));
    }
    return z;
}

template <int D>
cudaError_t launch(const PagedChunkParams &p, Sizes &z, cudaStream_t stream) {
    using L = Lay<D>;
    char *w = static_cast<char *>(p.workspace);
    z.plan.part_ml = reinterpret_cast<float2 *>(w);
    z.plan.part_o = reinterpret_cast<float *>(w + z.ml);
    CUtensorMap map_q{}, map_k{}, map_v{};
    const uint64_t row = (uint64_t)p.kv_heads * D * 2;
    const uint64_t dims[4] = {64, (uint64_t)p.num_pages * p.page_rows, D / 64, (uint64_t)p.kv_heads};
    const uint64_t strides[3] = {row, 128, D * 2};
    const uint32_t box_k[4] = {64, 64, 4, 1}, box_v[4] = {64, kKeys, 2, 1};
    const uint64_t dims_q[4] = {D, (uint64_t)p.q_heads, (uint64_t)p.k, (uint64_t)p.batch};
    const uint64_t strides_q[3] = {D * 2, (uint64_t)p.q_heads * D * 2,
                                   (uint64_t)p.k * p.q_heads * D * 2};
    const uint32_t box_q[4] = {64, (uint32_t)p.group, (uint32_t)z.plan.tokens, 1};
    if (!make_bf16_tensor_map(&map_q, p.q, 4, dims_q, strides_q, box_q, true) ||
        !make_bf16_tensor_map(&map_k, p.k_pages, 4, dims, strides, box_k, true) ||
        !make_bf16_tensor_map(&map_v, p.v_pages, 4, dims, strides, box_v, true))
        return cudaErrorInvalidValue;
    auto kernel = paged_chunk_kernel<D>;
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(1, std::memory_order_release);
    }
    e = launch_dependent(kernel, dim3((unsigned)(z.items * z.plan.splits * 2)), dim3(kThreads),
                         L::kAlloc, stream, p, z.plan, map_q, map_k, map_v);
    if (e != cudaSuccess || z.plan.splits == 1) return e;
    return launch_dependent(paged_chunk_merge_kernel<D>,
                            dim3((unsigned)(p.batch * p.k * p.q_heads)), dim3(D / 4), 0, stream, p,
                            z.plan);
}

}  // namespace

bool paged_chunk_supported(int head_dim) { return head_dim == 256 || head_dim == 512; }

size_t paged_chunk_workspace(int batch, int k, int q_heads, int kv_heads, int head_dim) {
    return sizes_of(batch, k, q_heads, kv_heads, head_dim).total;
}

cudaError_t launch_paged_chunk_attention(const PagedChunkParams &p, cudaStream_t stream) {
    Sizes z = sizes_of(p.batch, p.k, p.q_heads, p.kv_heads, p.head_dim);
    return p.head_dim == 256 ? launch<256>(p, z, stream) : launch<512>(p, z, stream);
}

}  // namespace carat
